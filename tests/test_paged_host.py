"""Refusals of the paged-cache entry points, on the host: the documented status comes back
before anything touches the device."""

import ctypes

import pytest

import online_activation_aware_b200 as ttq

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from online_activation_aware_b200 import build

    build.build()
    return ttq.load_library()


def P(v):
    return ctypes.c_void_p(v) if v else None


A, B, C, Q, O, W = (1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20, 6 << 20)  # fake addresses, never read


def plan_bytes(lib, *sizes):
    n = ctypes.c_size_t(0)
    assert lib.ttq_attention_plan_size(*sizes, ctypes.byref(n)) == OK
    return n.value


def test_plan_size(lib):
    n = ctypes.c_size_t(0)
    size = lambda *a: lib.ttq_attention_plan_size(*a, ctypes.byref(n))
    assert size(4, 100, 50, 40, 8, 128) == OK and n.value > 0 and n.value % 256 == 0
    assert lib.ttq_attention_plan_size(4, 100, 50, 40, 8, 128, None) == INVALID
    assert size(4, 100, 50, 40, 8, 96) == UNSUPPORTED
    assert size(4, 100, 50, 65, 1, 128) == UNSUPPORTED       # more than 64 heads a kv head
    assert size(4, 100, 50, 30, 8, 128) == INVALID
    assert size(4, 100, 101, 32, 8, 128) == INVALID          # max_new past the tokens
    assert size(4, 100, 0, 32, 8, 128) == INVALID
    assert size(0, 100, 50, 32, 8, 128) == INVALID
    assert size(4, 0, 0, 32, 8, 128) == INVALID
    assert size(65537, 1 << 20, 1, 32, 8, 128) == INVALID
    assert size(65536, 1 << 24, 1 << 24, 64, 1, 64) == OK


def test_plan_errors(lib):
    nb = plan_bytes(lib, 4, 100, 50, 32, 8, 128)

    def plan(start=A, length=B, prefix=0, window=0, seqs=4, ws=W, wsb=nb):
        return lib.ttq_attention_plan(P(start), P(length), P(prefix), window, seqs, 100, 50, 32, 8, 128, P(ws), wsb, None)

    assert plan(start=0) == INVALID
    assert plan(length=0) == INVALID
    assert plan(window=-1) == INVALID
    assert plan(seqs=0) == INVALID
    assert plan(ws=0) == WORKSPACE
    assert plan(wsb=nb - 256) == WORKSPACE
    assert plan(start=A + 2) == MISALIGNED
    assert plan(prefix=C + 2) == MISALIGNED
    assert plan(ws=W + 8) == MISALIGNED


def test_attention_errors(lib):
    nb = plan_bytes(lib, 4, 100, 50, 32, 8, 128)

    def att(q=Q, ld=4096, seqs=4, k=A, v=B, pages=100, page=32, table=C, width=9, cap=0.0, slopes=0, out=O, ws=W, wsb=nb,
            D=128):
        return lib.ttq_paged_attention(P(q), ld, seqs, 100, 50, 32, 8, D, P(k), P(v), pages, page, P(table), width,
                                       ctypes.c_float(cap), P(slopes), P(out), P(ws), wsb, None)

    assert att(q=0) == INVALID and att(out=0) == INVALID and att(k=0) == INVALID and att(table=0) == INVALID
    assert att(out=Q) == INVALID and att(k=B) == INVALID
    assert att(D=256) == UNSUPPORTED
    for page in (0, 8, 24, 48, 512):
        assert att(page=page) == UNSUPPORTED
    assert att(pages=0) == INVALID and att(pages=1 << 26) == INVALID and att(width=0) == INVALID
    assert att(ld=4088) == INVALID
    assert att(ld=4100) == MISALIGNED
    assert att(cap=-1.0) == INVALID and att(cap=float("nan")) == INVALID and att(cap=float("inf")) == INVALID
    assert att(ws=0) == WORKSPACE and att(wsb=16) == WORKSPACE
    assert att(cap=1e-38) == INVALID
    for name in ("q", "k", "v", "out", "ws"):
        assert att(**{name: 7 * (1 << 20) + 8}) == MISALIGNED
    for name in ("table", "slopes"):
        assert att(**{name: 7 * (1 << 20) + 2}) == MISALIGNED


def test_page_write_errors(lib):
    def app(qkv=Q, seqs=4, tokens=100, heads=32, D=128, eps=1e-6, rope=W, rows=64, k=A, v=B, pages=100, page=32, table=C,
            width=9, out=O, start=A + 4096):
        return lib.ttq_qk_norm_rope_paged(P(qkv), seqs, tokens, heads, 8, D, P(W), P(W), ctypes.c_float(eps), P(rope), rows,
                                          P(start), P(A), P(k), P(v), pages, page, P(table), width, P(out), None)

    assert app(D=96) == UNSUPPORTED and app(page=12) == UNSUPPORTED
    assert app(seqs=0) == INVALID and app(tokens=0) == INVALID and app(heads=0) == INVALID and app(rows=0) == INVALID
    assert app(eps=0.0) == INVALID and app(out=Q) == INVALID and app(v=A) == INVALID and app(start=0) == INVALID
    assert app(qkv=Q + 2) == MISALIGNED and app(out=O + 8) == MISALIGNED and app(start=A + 2) == MISALIGNED


def test_page_copy_and_remap_errors(lib):
    def copy(k=A, v=B, layers=2, pages=10, nb=4096, src=C, dst=Q, n=3):
        return lib.ttq_copy_pages(P(k), P(v), layers, pages, nb, P(src), P(dst), n, None)

    assert copy(k=0) == INVALID and copy(v=A) == INVALID and copy(src=0) == INVALID
    assert copy(layers=0) == INVALID and copy(pages=0) == INVALID and copy(n=0) == INVALID and copy(n=11) == INVALID
    assert copy(nb=0) == INVALID
    assert copy(nb=4104) == MISALIGNED and copy(k=A + 8) == MISALIGNED and copy(dst=Q + 2) == MISALIGNED

    def remap(table=A, n=10, m=B, pages=5, out=C):
        return lib.ttq_remap_pages(P(table), n, P(m), pages, P(out), None)

    assert remap(table=0) == INVALID and remap(n=0) == INVALID and remap(pages=0) == INVALID and remap(out=B) == INVALID
    assert remap(m=B + 2) == MISALIGNED


def test_logprob_errors(lib):
    def lp(x=A, dt=0, rows=8, vocab=1000, ld=1000, tok=B, top=5, a=C, e=Q, ids=O, tl=W):
        return lib.ttq_token_logprobs(P(x), dt, rows, vocab, ld, P(tok), top, P(a), P(e), P(ids), P(tl), None)

    assert lp(x=0) == INVALID and lp(tok=0) == INVALID and lp(a=0) == INVALID and lp(a=Q) == INVALID
    assert lp(dt=3) == UNSUPPORTED and lp(top=33) == UNSUPPORTED
    assert lp(vocab=4) == INVALID and lp(vocab=(1 << 20) + 1, ld=1 << 21) == INVALID
    assert lp(rows=0) == INVALID and lp(vocab=0) == INVALID and lp(ld=999) == INVALID and lp(top=-1) == INVALID
    assert lp(ids=0) == INVALID and lp(tl=0) == INVALID and lp(top=0) == INVALID
    assert lp(x=A + 1) == MISALIGNED and lp(x=A + 2, dt=2) == MISALIGNED
    assert lp(tok=B + 4) == MISALIGNED and lp(tl=W + 2) == MISALIGNED


def test_binding_refuses_wrong_tensors(lib):
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i = lambda *s: z(*s, dt=torch.int32)
    with pytest.raises(ValueError):
        ttq.copy_pages(z(4, 16, 2, 64), z(4, 16, 2, 64), i(1), i(1))          # CPU tensors
    with pytest.raises(ValueError):
        ttq.copy_pages(z(4, 16, 2, 64), z(5, 16, 2, 64), i(1), i(1))
    with pytest.raises(ValueError):
        ttq.copy_pages(z(16, 2, 64), z(16, 2, 64), i(1), i(1))
    with pytest.raises(ValueError):
        ttq.remap_pages(i(4), i(4))
    with pytest.raises(ValueError):
        ttq.token_logprobs(z(3, 8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        ttq.token_logprobs(z(8, 3).t(), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        ttq.token_logprobs(z(3, 8, dt=torch.float64), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ttq.TTQError):
        ttq.AttentionPlan(2, 4, 30, 8, 128, device="cpu")
    with pytest.raises(TypeError):
        ttq.remap_pages([1, 2], i(4))                                         # no tensor
    with pytest.raises(TypeError):
        ttq.token_logprobs(z(3, 8), torch.zeros(3, dtype=torch.int64), top="five")
    with pytest.raises(ValueError):
        ttq.qk_norm_rope_paged(z(3, 4 * 64), 2, 1, 64, z(64), z(64), 1e-6, z(9, 32, 2, dt=torch.float32), i(2), i(1),
                               z(4, 16, 1, 64), z(4, 16, 1, 64), i(1, 2))     # CPU tensors
