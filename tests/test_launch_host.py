"""The binding's launch from several threads at once: its two lookups of the current device and
stream are both there before either is used.  CPU only: torch is replaced."""
import sys
import types

import residual_add_rmsnorm_gb300 as rarn


def test_the_lookups_are_published_together(monkeypatch):
    monkeypatch.setattr(rarn, "_get_device", None)
    monkeypatch.setattr(rarn, "_raw_stream", None)

    class C:
        _cuda_getDevice = staticmethod(lambda: 0)

        @property
        def _cuda_getCurrentRawStream(self):
            # another thread that now sees _get_device would go on to call _raw_stream
            assert rarn._get_device is None or rarn._raw_stream is not None
            return lambda i: 7

    fake = types.SimpleNamespace(_C=C(), cuda=types.SimpleNamespace(current_device=None))
    monkeypatch.setitem(sys.modules, "torch", fake)
    got = []
    rarn._on(types.SimpleNamespace(index=0), "call", lambda *a: got.append(a) or 0, 1, 2)
    assert got == [(1, 2, 7)]
