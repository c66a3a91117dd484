"""What the expert layer's entry points refuse, and the sizes they name, on
the host alone: every refusal comes before anything is launched."""
import ctypes as C
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    from exact_quantile_selection_amd import build, qb

    if not os.path.exists(qb.LIB_PATH):
        build.build()
    return qb.lib()


def refused(L, status, words, rc):
    from exact_quantile_selection_amd import qb

    assert rc == getattr(qb, status), (rc, L.qb_last_error())
    assert words in L.qb_last_error().decode()


def test_sizes(L):
    from exact_quantile_selection_amd import qb

    assert qb.fp8_ld(1) == 128 and qb.fp8_ld(128) == 128 and qb.fp8_ld(129) == 256 and qb.fp8_ld(0) == 0
    assert qb.fp8_sld(1) == 4 and qb.fp8_sld(512) == 4 and qb.fp8_sld(513) == 8
    for N, E, B in ((1, 16, 1), (5003, 64, 41), (131072, 256, 32), (1 << 20, 256, 1)):
        n = L.qb_balance_workspace_bytes(N, E, B)
        assert 0 < n <= 16 * E * (B + N // 32 + 2)
    assert L.qb_balance_workspace_bytes(0, 16, 1) == qb.QB_EINVAL
    assert L.qb_balance_workspace_bytes(10, 48, 1) == qb.QB_EINVAL
    assert L.qb_dispatch_rows(16, 8, 256, 1) == 128
    assert L.qb_dispatch_rows(16, 8, 256, 128) == 16384          # 128 pairs, 128 experts at most
    assert L.qb_dispatch_rows(1000, 8, 64, 128) == (8000 + 64 * 127) // 128 * 128
    assert L.qb_dispatch_rows(0, 8, 64, 128) == 0
    assert L.qb_dispatch_workspace_bytes(1024, 8, 256) == 0      # one workgroup
    for N, K, E in ((1025, 8, 256), (32768, 8, 16), (1 << 20, 8, 256)):
        assert 0 < L.qb_dispatch_workspace_bytes(N, K, E) <= 8 * E * (N * K // 512 + 2)
    for rc in (L.qb_dispatch_rows(10, 0, 16, 1), L.qb_dispatch_rows(10, 2, 16, 0), L.qb_dispatch_rows(1 << 31, 2, 16, 1)):
        assert rc == qb.QB_EINVAL
    assert L.qb_dispatch_rows(10, 2, 257, 1) == qb.QB_EUNSUPPORTED
    with pytest.raises(qb.QBError):
        qb.qb_balance_workspace_bytes(10, 48)


def test_balance_refusals(L):
    def fwd(s=FAKE, b=FAKE, N=100, E=64, K=6, off=None, B=1, topk=FAKE, gate=None, count=None, weight=None, loss=None,
            ws=None, n=0):
        return L.qb_balance_forward(s, b, N, E, K, off, B, None, C.c_float(0.1), topk, gate, count, weight, loss, ws, n,
                                    None)

    need = L.qb_balance_workspace_bytes(100, 64, 1)
    refused(L, "QB_EINVAL", "s is NULL", fwd(s=None))
    refused(L, "QB_EINVAL", "16-byte aligned", fwd(s=FAKE + 4))
    refused(L, "QB_EINVAL", "N=0", fwd(N=0))
    refused(L, "QB_EINVAL", "2^30", fwd(N=(1 << 30) + 1))
    refused(L, "QB_EUNSUPPORTED", "E=48", fwd(E=48))
    refused(L, "QB_EINVAL", "K=64", fwd(K=64))
    refused(L, "QB_EINVAL", "K=0", fwd(K=0))
    refused(L, "QB_EUNSUPPORTED", "K=16", fwd(K=16))
    refused(L, "QB_EINVAL", "B=0", fwd(off=FAKE, B=0))
    refused(L, "QB_EINVAL", "seq_off", fwd(B=2))
    refused(L, "QB_EINVAL", "required", fwd(b=None))
    refused(L, "QB_EINVAL", "required", fwd(topk=None))
    refused(L, "QB_EINVAL", "ws_bytes=0", fwd(loss=FAKE))
    refused(L, "QB_EINVAL", "ws_bytes", fwd(count=FAKE, ws=FAKE, n=need - 1))
    refused(L, "QB_EINVAL", "ws must be 16-byte", fwd(count=FAKE, ws=FAKE + 8, n=need))
    refused(L, "QB_EINVAL", "weight must be 16-byte", fwd(weight=FAKE + 4, ws=FAKE, n=need))
    refused(L, "QB_EINVAL", "4-byte aligned", fwd(gate=FAKE + 2))
    refused(L, "QB_EINVAL", "4-byte aligned", fwd(off=FAKE + 1))

    def bwd(s=FAKE, topk=FAKE, N=100, E=64, K=6, off=None, B=1, weight=FAKE, dloss=None, dgate=FAKE, dx=FAKE):
        return L.qb_balance_backward(s, topk, N, E, K, off, B, None, weight, dloss, dgate, dx, None)

    refused(L, "QB_EINVAL", "nothing to differentiate", bwd(weight=None, dgate=None))
    refused(L, "QB_EINVAL", "needs topk", bwd(topk=None))
    refused(L, "QB_EINVAL", "dlogits", bwd(dx=None))
    refused(L, "QB_EINVAL", "16-byte", bwd(dx=FAKE + 8))
    refused(L, "QB_EINVAL", "16-byte", bwd(weight=FAKE + 8))
    refused(L, "QB_EINVAL", "4-byte", bwd(dloss=FAKE + 2))
    refused(L, "QB_EUNSUPPORTED", "E=512", bwd(E=512))


def test_exchange_refusals(L):
    def disp(topk=FAKE, N=2000, K=8, E=64, align=128, off=FAKE, R=None, src=FAKE, pos=FAKE, ws=FAKE, n=1 << 20):
        R = L.qb_dispatch_rows(2000, 8, 64, 128) if R is None else R
        return L.qb_dispatch(topk, N, K, E, align, off, R, src, pos, ws, n, None)

    refused(L, "QB_EUNSUPPORTED", "E=300", disp(E=300))
    refused(L, "QB_EINVAL", "align=0", disp(align=0))
    refused(L, "QB_EINVAL", "N=-1", disp(N=-1))
    refused(L, "QB_EINVAL", "N K < 2^31", disp(N=1 << 29))
    refused(L, "QB_EINVAL", "qb_dispatch_rows", disp(R=16000))
    for k in ("topk", "off", "src", "pos"):
        refused(L, "QB_EINVAL", "required", disp(**{k: None}))
        refused(L, "QB_EINVAL", "4-byte", disp(**{k: FAKE + 2}))
    refused(L, "QB_EINVAL", "qb_dispatch_workspace_bytes", disp(ws=None))
    refused(L, "QB_EINVAL", "ws_bytes=16", disp(n=16))
    refused(L, "QB_EINVAL", "ws must be 16-byte", disp(ws=FAKE + 4))

    def comb(rows=FAKE, R=100, pos=FAKE, gate=None, N=10, K=2, H=64, out=FAKE):
        return L.qb_combine(rows, R, pos, gate, N, K, H, out, None)

    refused(L, "QB_EINVAL", "H=0", comb(H=0))
    refused(L, "QB_EINVAL", "K=0", comb(K=0))
    refused(L, "QB_EINVAL", "2^24", comb(N=(1 << 24) + 1))
    refused(L, "QB_EINVAL", "required", comb(rows=None))
    refused(L, "QB_EINVAL", "2-byte", comb(out=FAKE + 1))
    refused(L, "QB_EINVAL", "4-byte", comb(gate=FAKE + 2))
    assert comb(N=0, pos=None, out=None) == 0                    # no token: nothing to do

    def back(dout=FAKE, rows=FAKE, R=100, pos=FAKE, src=FAKE, gate=None, N=10, K=2, H=64, drows=FAKE, dgate=None):
        return L.qb_combine_backward(dout, rows, R, pos, src, gate, N, K, H, drows, dgate, None)

    refused(L, "QB_EINVAL", "required", back(dout=None))
    refused(L, "QB_EINVAL", "required", back(src=None))
    refused(L, "QB_EINVAL", "needs rows", back(rows=None, dgate=FAKE))
    refused(L, "QB_EINVAL", "2-byte", back(drows=FAKE + 1))
    refused(L, "QB_EINVAL", "4-byte", back(dgate=FAKE + 1))


def test_fp8_refusals(L):
    for fn in (L.qb_fp8_quantize, L.qb_fp8_quantize_cols):
        q = lambda x=FAKE, Mx=10, src=None, M=10, c=100, o=FAKE, s=FAKE: fn(x, Mx, src, M, c, o, s, None)  # noqa: E731
        refused(L, "QB_EINVAL", "Mx=11", q(Mx=11))               # another number of rows needs row_src
        refused(L, "QB_EINVAL", "M=-1", q(M=-1))
        refused(L, "QB_EINVAL", "2^22", q(M=(1 << 22) + 1, Mx=(1 << 22) + 1))
        refused(L, "QB_EINVAL", "C=0", q(c=0))
        refused(L, "QB_EINVAL", "required", q(x=None))
        refused(L, "QB_EINVAL", "required", q(s=None))
        refused(L, "QB_EINVAL", "16-byte", q(o=FAKE + 8))
        refused(L, "QB_EINVAL", "16-byte", q(s=FAKE + 2))
        refused(L, "QB_EINVAL", "2-byte", q(x=FAKE + 1))
        refused(L, "QB_EINVAL", "4-byte", q(src=FAKE + 2))
        assert q(x=None, Mx=0, M=0) == 0

    w = lambda x=FAKE, g=2, n=10, c=10, q=FAKE, s=FAKE, t=FAKE, ts=FAKE: (  # noqa: E731
        L.qb_fp8_quantize_weight(x, g, n, c, q, s, t, ts, None))
    refused(L, "QB_EUNSUPPORTED", "G=257", w(g=257))
    refused(L, "QB_EINVAL", "both or neither", w(ts=None))
    refused(L, "QB_EINVAL", "required", w(x=None))
    refused(L, "QB_EINVAL", "16-byte", w(t=FAKE + 1))

    p = lambda x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, m=10, n=10, c=10, off=None, g=1, ex=0, y=FAKE: (  # noqa: E731
        L.qb_fp8_product(x, xs, w, ws, m, n, c, off, g, ex, y, None))
    refused(L, "QB_EINVAL", "exact=2", p(ex=2))
    refused(L, "QB_EINVAL", "need off", p(g=2))
    refused(L, "QB_EUNSUPPORTED", "G=0", p(g=0, off=FAKE))
    refused(L, "QB_EINVAL", "N=0", p(n=0))
    for k in ("x", "xs", "w", "ws", "y"):
        refused(L, "QB_EINVAL", "required", p(**{k: None}))
        refused(L, "QB_EINVAL", "aligned", p(**{k: FAKE + 1}))
    refused(L, "QB_EINVAL", "4-byte", p(off=FAKE + 2))
    assert p(m=0, x=None) == 0

    d = lambda a=FAKE, s=FAKE, b=FAKE, t=FAKE, m=10, n=10, c=10, off=None, g=1, o=FAKE: (  # noqa: E731
        L.qb_fp8_weight_grad(a, s, b, t, m, n, c, off, g, o, None))
    refused(L, "QB_EINVAL", "need off", d(g=2))
    for k in ("a", "s", "b", "t", "o"):
        refused(L, "QB_EINVAL", "required", d(**{k: None}))
        refused(L, "QB_EINVAL", "aligned", d(**{k: FAKE + 1}))
    refused(L, "QB_EINVAL", "M=4194305", d(m=(1 << 22) + 1))


def test_the_binding_names_a_wrong_tensor():
    import torch

    from exact_quantile_selection_amd import qb

    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        qb.qb_fp8_quantize(x, x, x)
    with pytest.raises(ValueError, match="rows must be a GPU tensor"):
        qb.qb_combine(x, torch.zeros((4, 2), dtype=torch.int32), x)
    with pytest.raises(ValueError, match="topk must be a GPU tensor"):
        qb.qb_dispatch(torch.zeros((4, 2), dtype=torch.int32), 16, 1, x, x, x)


def test_the_binding_refuses_what_is_no_gpu_tensor(L):
    """The compiled binding turns wrong arguments into the errors that the
    rest of the binding raises, before any call of the library."""
    import torch

    from exact_quantile_selection_amd import qb

    s, b = torch.zeros((4, 16)), torch.zeros(16)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    for bad in (s, None, 3, "s"):
        with pytest.raises(ValueError, match="s (must be a GPU tensor|is required)"):
            qb.qb_balance_forward(bad, b, 2, ids, stream=Stream())
    with pytest.raises(ValueError, match="rows must be a GPU tensor"):
        qb.qb_combine(s.to(torch.bfloat16), ids, s.to(torch.bfloat16), stream=Stream())
    with pytest.raises(ValueError, match="row_src must be a GPU tensor|x must be a GPU tensor"):
        qb.qb_fp8_quantize(s.to(torch.bfloat16), None, None, row_src=ids, stream=Stream())
    with pytest.raises(ValueError, match="w is required"):
        qb.qb_fp8_quantize_weight(None, None, None, stream=Stream())
    with pytest.raises(TypeError, match="13 arguments"):
        qb._calls().balance_forward(s, b)


class Stream:
    """Stands for a stream where nothing is launched."""
    cuda_stream = 0
