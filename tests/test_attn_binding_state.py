"""The attention operators' binding: its first use from several threads, and the
streams it refuses (no GPU needed: calls stop before the library)."""
import threading
import time
from types import SimpleNamespace

import pytest

import block_quantized_matmul_amd as qmm
from block_quantized_matmul_amd import attn


class _Calls(dict):
    """Functions by name, each stored once and with its argument types set: other threads use an entry as soon as it is
    here, and without the types a pointer would be passed as an int."""

    def __setitem__(self, name, function):
        assert name not in self, f"{name} replaced"
        assert function.argtypes and function.restype is attn._i32, f"{name} stored before its types"
        time.sleep(0.01)
        super().__setitem__(name, function)


def test_first_use_from_several_threads(monkeypatch):
    attn._lib()
    loaded = qmm.lib()

    def slow_lib():
        time.sleep(0.05)  # every thread gets here before one is done
        return loaded

    monkeypatch.setattr(attn, "_ready", None)
    monkeypatch.setattr(attn, "_calls", _Calls())
    monkeypatch.setattr(attn._qmm, "lib", slow_lib)
    failed, start = [], threading.Barrier(4)

    def first_call():
        try:
            start.wait()
            assert attn._lib() is loaded
            assert sorted(attn._calls) == ["qmm_attn_prompt", "qmm_attn_shared", "qmm_norm_rope"]
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=first_call) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_a_stream_of_another_gpu_is_refused(monkeypatch):
    """Also where its handle is that of the tensors' current stream, as those of two GPUs' default streams are."""
    attn._lib()
    monkeypatch.setattr(attn, "torch", SimpleNamespace(_C=SimpleNamespace(_cuda_getCurrentRawStream=lambda device: 0)))
    tensor = SimpleNamespace(get_device=lambda: 0)

    def stream(index, handle):
        return SimpleNamespace(device=SimpleNamespace(index=index), cuda_stream=handle)

    for handle in (0, 77):
        with pytest.raises(ValueError, match="stream"):
            attn._Place(stream(1, handle), ("X",), [tensor])
    place = attn._Place(stream(0, 0), ("X",), [tensor])
    assert place.handle == 0 and place.foreign is None
    own = stream(0, 77)
    place = attn._Place(own, ("X",), [tensor])
    assert place.handle == 77 and place.foreign is own
