"""What the bf16 and 4-bit products, the orthogonalised update and the layer that
uses them refuse, and the sizes they name, on the host alone: every refusal comes
before anything is launched."""
import inspect
import os

import pytest

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

    assert qb.fp4_ld(1) == 128 and qb.fp4_ld(256) == 128 and qb.fp4_ld(257) == 256 and qb.fp4_ld(0) == 0
    assert qb.fp4_sld(1) == 8 and qb.fp4_sld(256) == 8 and qb.fp4_sld(257) == 16
    grad = L.qb_bf16_weight_grad_workspace_bytes
    assert grad(131072, 1024, 2048, 64) == 0             # tiles enough
    assert grad(100, 128, 128, 1) == 0                   # a short sum
    assert grad(131072, 128, 128, 1) == 16 * 4 * 128 * 128
    for M, N, C, G in ((131072, 128, 128, 1), (1 << 22, 1, 1, 1), (65536, 1000, 2000, 1), (9000, 64, 72, 2), (99999, 300, 300, 7)):
        assert 0 <= grad(M, N, C, G) <= 32 << 20
    assert grad(10, 0, 10, 1) == qb.QB_EINVAL and grad(10, 10, 10, 257) == qb.QB_EUNSUPPORTED
    ortho = L.qb_orthogonalize_workspace_bytes
    for G, N, C in ((1, 1, 1), (5, 301, 165), (64, 1024, 2048), (1, 65536, 8)):
        assert 0 < ortho(G, N, C) <= 20 * G * (N + 128) * (C + 128) + (1 << 20)
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (65536, 1, 1), (1, 65537, 1), (1, 1, 65537)):
        assert ortho(*bad) == qb.QB_EINVAL
    with pytest.raises(qb.QBError):
        qb.qb_orthogonalize_workspace_bytes(0, 1, 1)
    with pytest.raises(qb.QBError):
        qb.qb_bf16_weight_grad_workspace_bytes(-1, 1, 1)


def test_bf16_refusals(L):
    p = lambda x=FAKE, Mx=10, src=None, M=10, w=FAKE, n=10, c=10, off=None, g=1, t=0, y=FAKE: (  # noqa: E731
        L.qb_bf16_product(x, Mx, src, M, w, n, c, off, g, t, y, None))
    refused(L, "QB_EINVAL", "Mx=11", p(Mx=11))
    refused(L, "QB_EINVAL", "Mx=-1", p(Mx=-1, src=FAKE))
    refused(L, "QB_EINVAL", "Mx=4194305", p(Mx=(1 << 22) + 1, src=FAKE))
    refused(L, "QB_EINVAL", "M=4194305", p(M=(1 << 22) + 1))
    refused(L, "QB_EINVAL", "N=0", p(n=0))
    refused(L, "QB_EINVAL", "C=0", p(c=0))
    refused(L, "QB_EINVAL", "need off", p(g=2))
    refused(L, "QB_EUNSUPPORTED", "G=257", p(g=257, off=FAKE))
    refused(L, "QB_EINVAL", "transposed=2", p(t=2))
    for k in ("x", "w", "y"):
        refused(L, "QB_EINVAL", "required", p(**{k: None}))
        refused(L, "QB_EINVAL", "2-byte", p(**{k: FAKE + 1}))
    refused(L, "QB_EINVAL", "4-byte", p(off=FAKE + 2))
    refused(L, "QB_EINVAL", "4-byte", p(src=FAKE + 2))
    assert p(M=0, Mx=0, x=None, w=None, y=None) == 0
    assert p(M=0, Mx=5) == 0                             # (an array of no numbers may be null)

    d = lambda dy=FAKE, x=FAKE, Mx=3000, src=None, M=3000, n=10, c=10, off=None, g=1, o=FAKE, ws=None, b=0: (  # noqa: E731
        L.qb_bf16_weight_grad(dy, x, Mx, src, M, n, c, off, g, o, ws, b, None))
    refused(L, "QB_EINVAL", "Mx=3001", d(Mx=3001))
    refused(L, "QB_EINVAL", "need off", d(g=2))
    refused(L, "QB_EINVAL", "M=-1", d(M=-1))
    for k in ("dy", "x", "o"):
        refused(L, "QB_EINVAL", "required", d(**{k: None}))
        refused(L, "QB_EINVAL", "aligned", d(**{k: FAKE + 1}))
    need = L.qb_bf16_weight_grad_workspace_bytes(3000, 10, 10, 1)
    assert need > 0
    refused(L, "QB_EINVAL", "qb_bf16_weight_grad_workspace_bytes", d(ws=FAKE, b=need - 1))
    refused(L, "QB_EINVAL", "ws must be 16-byte", d(ws=FAKE + 8, b=need))
    refused(L, "QB_EINVAL", "4-byte", d(off=FAKE + 2))
    refused(L, "QB_EINVAL", "4-byte", d(src=FAKE + 1))


def test_fp4_refusals(L):
    q = lambda x=FAKE, Mx=10, src=None, M=10, c=100, o=FAKE, s=FAKE: (  # noqa: E731
        L.qb_fp4_quantize(x, Mx, src, M, c, o, s, None))
    refused(L, "QB_EINVAL", "Mx=11", q(Mx=11))
    refused(L, "QB_EINVAL", "M=-1", q(M=-1))
    refused(L, "QB_EINVAL", "C=0", q(c=0))
    for k in ("x", "o", "s"):
        refused(L, "QB_EINVAL", "required", q(**{k: None}))
    refused(L, "QB_EINVAL", "2-byte", q(x=FAKE + 1))
    refused(L, "QB_EINVAL", "16-byte", q(o=FAKE + 8))
    refused(L, "QB_EINVAL", "8-byte", q(s=FAKE + 4))
    refused(L, "QB_EINVAL", "4-byte", q(src=FAKE + 2))
    assert q(x=None, Mx=0, M=0) == 0

    w = lambda x=FAKE, g=2, n=10, c=10, q=FAKE, s=FAKE, t=FAKE, ts=FAKE: (  # noqa: E731
        L.qb_fp4_quantize_weight(x, g, n, c, q, s, t, ts, None))
    refused(L, "QB_EUNSUPPORTED", "G=257", w(g=257))
    refused(L, "QB_EINVAL", "both or neither", w(ts=None))
    refused(L, "QB_EINVAL", "required", w(x=None))
    refused(L, "QB_EINVAL", "16-byte", w(t=FAKE + 8))
    refused(L, "QB_EINVAL", "8-byte", w(ts=FAKE + 4))
    refused(L, "QB_EINVAL", "4-byte", w(x=FAKE + 2))

    p = lambda x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, m=10, n=10, c=10, off=None, g=1, y=FAKE: (  # noqa: E731
        L.qb_fp4_product(x, xs, w, ws, m, n, c, off, g, y, None))
    refused(L, "QB_EINVAL", "need off", p(g=2))
    refused(L, "QB_EUNSUPPORTED", "G=0", p(g=0, off=FAKE))
    refused(L, "QB_EINVAL", "N=0", p(n=0))
    for k in ("x", "xs", "w", "ws", "y"):
        refused(L, "QB_EINVAL", "required", p(**{k: None}))
        refused(L, "QB_EINVAL", "aligned", p(**{k: FAKE + 1}))
    refused(L, "QB_EINVAL", "4-byte", p(off=FAKE + 2))
    assert p(m=0, x=None) == 0


def test_orthogonalize_refusals(L):
    need = L.qb_orthogonalize_workspace_bytes(2, 10, 20)
    o = lambda x=FAKE, g=2, n=10, c=20, steps=5, out=FAKE, ws=FAKE, b=need: (  # noqa: E731
        L.qb_orthogonalize(x, g, n, c, steps, 1.5, -0.5, 0.0, out, ws, b, None))
    refused(L, "QB_EINVAL", "G=0", o(g=0))
    refused(L, "QB_EINVAL", "N=0", o(n=0))
    refused(L, "QB_EINVAL", "C=65537", o(c=65537))
    refused(L, "QB_EINVAL", "steps=0", o(steps=0))
    refused(L, "QB_EINVAL", "steps=65", o(steps=65))
    refused(L, "QB_EINVAL", "required", o(x=None))
    refused(L, "QB_EINVAL", "required", o(out=None))
    refused(L, "QB_EINVAL", "ws_bytes=0", o(ws=None))
    refused(L, "QB_EINVAL", "qb_orthogonalize_workspace_bytes", o(b=need - 1))
    refused(L, "QB_EINVAL", "ws must be 16-byte", o(ws=FAKE + 8))
    refused(L, "QB_EINVAL", "2-byte", o(out=FAKE + 1))
    refused(L, "QB_EINVAL", "4-byte", o(x=FAKE + 2))


def test_the_binding_names_a_wrong_tensor():
    import torch

    from exact_quantile_selection_amd import qb

    x, u = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((4, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        qb.qb_bf16_product(x, x, x)
    with pytest.raises(ValueError, match="dy must be a GPU tensor"):
        qb.qb_bf16_weight_grad(x, x, x)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        qb.qb_fp4_quantize(x, u, u)
    with pytest.raises(ValueError, match="w is required"):
        qb.qb_fp4_quantize_weight(None, u, u)
    with pytest.raises(ValueError, match="xq must be a GPU tensor"):
        qb.qb_fp4_product(u, u, u, u, x)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        qb.qb_orthogonalize(x.float(), x, u)
    with pytest.raises(ValueError, match="x must be"):
        qb.qb_orthogonalize(x.float()[0], x, u)
    with pytest.raises(TypeError, match="7 arguments"):
        qb._calls().bf16_product(x, x)


def test_the_layer_says_how_its_matrices_may_be_held():
    import torch

    from exact_quantile_selection_amd.expert_layer import ExpertLayer

    assert inspect.signature(ExpertLayer).parameters["held"].default == "e4m3"
    wr, w = torch.zeros((32, 64), dtype=torch.bfloat16), torch.zeros((32, 16, 64))
    with pytest.raises(ValueError, match="held='fp16'"):
        ExpertLayer(wr, w, 2, 10, held="fp16")
    with pytest.raises(ValueError, match="exact=False"):
        ExpertLayer(wr, w, 2, 10, held="bf16", exact=False)
