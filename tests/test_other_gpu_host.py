"""Tensors of a GPU that is not the current one, on the host: every entry point makes the tensors' GPU the
current one while the library runs, for a default stream's handle means the current GPU's. The
library, the GPUs and the tensors' place are stand-ins; nothing is launched."""

import pytest
import torch

import trellis_quantized_linear_tf_amd as tq
from trellis_quantized_linear_tf_amd import _lib

K, N, BITS = 256, 384, 4
f16, bf, i32 = torch.float16, torch.bfloat16, torch.int32


class Far(torch.Tensor):
    """A tensor on the host that says it is on GPU 1."""

    is_cuda = True

    def get_device(self):
        return 1


def far(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Far)


class Machine:
    def __init__(self, status):
        self.now, self.status, self.calls = 0, status, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace"):
                return 16
            if name == "tf_exl3_status_string":
                return b"refused"
            self.calls.append((name, self.now, args[-1]))
            return self.status
        return call

    def guard(self, device):
        machine = self

        class Guard:
            def __enter__(self):
                self.before, machine.now = machine.now, int(device)

            def __exit__(self, *exc):
                machine.now = self.before

        return Guard()


@pytest.fixture
def machine(monkeypatch, request):
    m = Machine(getattr(request, "param", 0))
    monkeypatch.setattr(_lib, "_lib", m)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: m.now)
    monkeypatch.setattr(torch.cuda, "device", m.guard)
    return m


def stream():
    return far(K * N * BITS // 32, dtype=i32)


def attention():
    q, k = far(2, 3, 4, 64, dtype=bf), far(2, 3, 2, 64, dtype=bf)
    cache = far(5, 16, 2, 64, dtype=bf)
    return q, k, k.clone(), far(2, 3, dtype=torch.int64), cache, cache.clone(), far(2, 2, dtype=i32), far(2, dtype=i32)


def drafts():
    return far(2, 3, 50), far(2, 3, dtype=i32), far(2, 3, dtype=i32), far(2, 2, 50), far(2, 3)


def rows():
    return far(3, 50), far(3, 5, dtype=i32), far(3, 5), far(3)


def append():
    _, k, v, _, kc, vc, table, lengths = attention()
    tq.cache_append(k, v, kc, vc, table, lengths)


CALLS = {
    "rot_in": lambda: tq.rot_in(far(2, K), far(K, dtype=f16)),
    **{f"linear {e}": lambda e=e: tq.linear(far(2, K, dtype=f16), stream(), far(N, dtype=f16), BITS, N, engine=e)
       for e in _lib.ENGINES},
    "project": lambda: tq.project(far(2, K), far(K, dtype=f16), stream(), far(N, dtype=f16), BITS, N),
    "repack_strips": lambda: tq.repack_strips(stream(), BITS, K, N),
    "decode_states": lambda: tq.debug_decode_states(far(64, dtype=torch.int16)),
    "decode_tiles": lambda: tq.debug_decode_tiles(stream(), BITS, K, N),
    "split": lambda: tq.debug_linear_split(far(2, K, dtype=f16), stream(), far(N, dtype=f16), BITS, N, split=0),
    "mfma split": lambda: _lib.debug_linear_mfma_split(far(2, K, dtype=f16), stream(), far(N, dtype=f16), BITS, N, split=0),
    "calib_copy": lambda: tq.calib_copy(far(64), far(64)),
    "calib_stream_read": lambda: tq.calib_stream_read(far(64), far(256, dtype=i32)),
    "tree_attention": lambda: tq.tree_attention(*attention()),
    "cache_append": append,
    "verify_tree": lambda: tq.verify_tree(drafts()[0], *drafts()[1:3], drafts()[4]),
    "verify_chain": lambda: tq.verify_chain(drafts()[0], drafts()[1], drafts()[3], drafts()[4]),
    "distill": lambda: tq.distill(*rows()),
    "distill_loss": lambda: tq.distill_loss(*rows()[:3]),
    "distill_grad": lambda: tq.distill_grad(*rows()),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_gpu_is_current_during_the_call(machine, name):
    CALLS[name]()
    assert [c[1:] for c in machine.calls] == [(1, 1001)]  # on GPU 1, its stream
    assert machine.now == 0


@pytest.mark.parametrize("machine", [-9], indirect=True)
@pytest.mark.parametrize("name", ["project", "tree_attention", "distill"])
def test_the_current_gpu_is_restored_after_a_refusal(machine, name):
    with pytest.raises(tq.Exl3Error):
        CALLS[name]()
    assert machine.calls[0][1] == 1 and machine.now == 0
