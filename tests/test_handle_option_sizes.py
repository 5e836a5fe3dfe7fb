"""The sizes of what is set on a handle, which the library reads without knowing them: calls that
would read another number of values are refused by the binding."""
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture
def G(monkeypatch):
    """The binding with a library that does nothing, and a handle of 2 groups of top 2."""
    from moe_query_head_b200 import gqe
    calls = []

    status_str = gqe.lib.gqe_status_str

    class Lib:
        gqe_status_str = staticmethod(status_str)

        def __getattr__(self, name):
            def fn(*args):
                if name == "gqe_create":
                    args[0]._obj.value = 0x7000
                calls.append(name)
                return 0
            return fn

    monkeypatch.setattr(gqe, "lib", Lib())
    monkeypatch.setattr(gqe, "_set_on", {}, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    gqe.calls = calls
    yield gqe
    del gqe.calls


class Fake:
    """A device tensor as the binding sees it."""

    def __init__(self, n, dtype=torch.int32, index=0):
        self.n, self.dtype, self.index = n, dtype, index

    def numel(self):
        return self.n

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


F32, F64 = torch.float32, torch.float64
ST = SimpleNamespace(cuda_stream=0)
X = Fake(1)


def handle(G):
    return G.gqe_create(64, 8, 2, 2, 16, G.GQE_BF16, 64)


def forward(G, h, B, T, shared=True):
    G.gqe_forward(h, X, B, T, X, X, X, X, X if shared else None, X, 8, 2, 2, 16, 0, 1, X, stream=ST)


def decode(G, h, B, shared=True):
    G.gqe_decode(h, X, B, X, X, 9, X, X, X, X, X, X if shared else None, X, 8, 2, 2, 16, 0, X, stream=ST)


def refused(G, fn, *a, **kw):
    n = len(G.calls)
    with pytest.raises(G.GQEError) as e:
        fn(*a, **kw)
    assert e.value.status == G.GQE_ERR_INVALID_ARG and len(G.calls) == n


def test_intervals(G):
    h = handle(G)
    forward(G, h, 2, 5)
    G.gqe_set_scores(h, softcap=3.0)
    forward(G, h, 2, 5)
    for name in ("key_begin", "key_end"):
        G.gqe_set_scores(h, **{name: Fake(10)})
        forward(G, h, 2, 5)
        forward(G, h, 1, 10)
        for B, T in ((2, 6), (1, 5), (3, 5)):
            refused(G, forward, G, h, B, T)
    G.gqe_set_scores(h, key_begin=Fake(2))  # of a decode step
    decode(G, h, 2)
    refused(G, forward, G, h, 2, 5)
    refused(G, decode, G, h, 3)
    G.gqe_set_scores(h, key_end=Fake(10))  # a decode step reads no ends
    decode(G, h, 3)
    G.gqe_set_scores(h)
    forward(G, h, 7, 5)
    G.gqe_destroy(h)


def test_slopes_follow_the_streams(G):
    h = handle(G)
    G.gqe_set_scores(h, slopes=Fake(5, F32))
    forward(G, h, 1, 4)
    decode(G, h, 3)
    refused(G, forward, G, h, 1, 4, shared=False)
    refused(G, decode, G, h, 3, shared=False)
    G.gqe_set_group_range(h, 0, 1)
    refused(G, forward, G, h, 1, 4)
    G.gqe_set_scores(h, slopes=Fake(3, F32))
    forward(G, h, 1, 4)
    G.gqe_set_scores(h, slopes=Fake(2, F32))
    refused(G, forward, G, h, 1, 4)
    forward(G, h, 1, 4, shared=False)


def test_positions(G):
    h = handle(G)
    G.gqe_set_qk_transform(h, 16, inv_freq=Fake(8, F64), positions=Fake(12))
    forward(G, h, 3, 4)
    refused(G, forward, G, h, 3, 5)
    decode(G, h, 5)  # at the caches' rows
    G.gqe_set_qk_transform(h, 16, inv_freq=Fake(8, F64))
    forward(G, h, 3, 5)
    G.gqe_set_qk_transform(h, 16, inv_freq=Fake(8, F64), positions=Fake(12))
    G.gqe_set_qk_transform(h)
    forward(G, h, 3, 5)


def test_devices_and_types(G):
    h = handle(G)
    refused(G, G.gqe_set_scores, h, slopes=Fake(5, F32, 1))  # not the handle's device
    refused(G, G.gqe_set_scores, h, slopes=Fake(5, F32, -1))
    refused(G, G.gqe_set_scores, h, key_begin=Fake(5, torch.int64))
    refused(G, G.gqe_set_qk_transform, h, 16, q_weight=Fake(16, F32, 1))
    refused(G, G.gqe_set_qk_transform, h, 16, q_weight=Fake(15, F32))
    refused(G, G.gqe_set_qk_transform, h, 16, inv_freq=Fake(8, F32))
    # a handle made and destroyed elsewhere is not known and not checked
    G.gqe_destroy(h)
    forward(G, h, 2, 5)


@pytest.mark.gpu
def test_on_a_handle():
    """The same on the GPU: the refused calls launch nothing, and the layer goes on."""
    from moe_query_head_b200 import gqe
    from moe_query_head_b200 import workloads as W
    from tests.gqe_testlib import GpuRun
    wl = W.WORKLOADS["main_b8_t2048"].with_(B=2, T=70)
    run = GpuRun(W.generate(wl)).forward()
    plain = run.out.clone()
    zeros = torch.zeros(wl.M, dtype=torch.int32, device="cuda")
    gqe.gqe_set_scores(run.h, key_begin=zeros[:wl.B])
    run.out.fill_(7.0)
    with pytest.raises(gqe.GQEError):
        run.forward()
    gqe.gqe_set_scores(run.h, slopes=torch.zeros(wl.G * wl.k, device="cuda"))
    with pytest.raises(gqe.GQEError):
        run.forward()
    assert (run.out == 7.0).all()
    gqe.gqe_set_scores(run.h, key_begin=zeros, slopes=torch.zeros(wl.G * wl.k + 1, device="cuda"))
    run.forward()
    # the same scores from another kernel: bf16 weights on both sides
    a, b = run.out.double(), plain.double()
    assert ((a - b).norm() / b.norm()) <= 1e-2
    run.close()
