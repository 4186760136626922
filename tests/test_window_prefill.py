"""hata_window_prefill against attention in 64 bits: lengths from one to thousands, windows and sinks that end inside
tiles, every kind of head group, rows past the end, refusals."""
import ctypes

import pytest
import torch

from attention_testlib import attend, close

D = 128


@pytest.fixture(scope="module")
def H():
    import hash_aware_top_b200 as H

    return H


def case(H, Hq, Hkv, max_seq, lens, window, sink, seed=0, scale_q=1.0, rows=None):
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = H.dims_for(B, Hq, Hkv, D, 128, max_seq, "bf16")
    q = (scale_q * torch.randn(B, Hq, max_seq, D, generator=g, device="cuda")).bfloat16()
    K, V = (torch.randn(B, Hkv, max_seq, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    for b, L in enumerate(lens):
        K[b, :, L:], V[b, :, L:], q[b, :, L:] = float("nan"), float("nan"), float("nan")
    out = torch.full_like(q, 9.0)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    H.hata_window_prefill(d, q, K, V, lens_d, window, sink, 0.0, out, ws)
    assert H.hata_read_device_status(ws) == 0
    for b, L in enumerate(lens):
        assert bool((out[b, :, L:] == 9.0).all())
        t = torch.arange(L, device="cuda") if rows is None or L <= rows else torch.randperm(L, generator=g, device="cuda")[:rows]
        s = torch.arange(L, device="cuda")
        sees = (s[None] <= t[:, None]) & ((s[None] < sink) | (s[None] > t[:, None] - window))
        for h in range(Hq):
            if L:
                want, absv, qk = attend(q[b, h, t], K[b, h // (Hq // Hkv), :L], V[b, h // (Hq // Hkv), :L], sees)
                close(out[b, h, t], want, absv, qk, min(L, window + sink), torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 2, 63, 64, 65, 127, 128, 129, 256, 300, 513])
def test_lengths(H, L):
    case(H, 4, 1, L, [L], 100, 3, seed=L)
    case(H, 2, 2, L, [L, (L + 1) // 2], 64, 0, seed=L)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 5), (2, 128), (127, 0), (128, 1), (129, 129), (333, 130), (10**9, 0),
                                         (5, 10**9), (700, 700), (100, 300), (64, 9), (70, 136), (200, 640), (2**31 - 1, 2**31 - 1)])
def test_windows(H, window, sink):
    case(H, 4, 2, 1025, [1025, 0, 700, 1], window, sink, seed=window % 997 + sink % 997)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (4, 1), (6, 2), (8, 1), (12, 4), (16, 1), (10, 2), (7, 7)])
def test_heads(H, Hq, Hkv):
    case(H, Hq, Hkv, 777, [777, 250], 200, 17, seed=Hq)


@pytest.mark.gpu
def test_long(H):
    case(H, 8, 2, 9000, [9000, 8191], 1500, 4, rows=300)


@pytest.mark.gpu
def test_many_short_prompts(H):
    case(H, 4, 2, 200, [(b * 53) % 201 for b in range(40)], 50, 2, rows=50)


@pytest.mark.gpu
def test_sharp_softmax(H):
    """Queries thirty times as large: maxima move often, and O is rescaled."""
    case(H, 4, 1, 1500, [1500], 600, 2, scale_q=30.0)


@pytest.mark.gpu
def test_wide_window_is_causal_prefill(H):
    """A window of the whole prompt sees what hata_prefill_attention sees; each rounds p and the result once."""
    L = 1000
    d = H.dims_for(1, 8, 2, D, 128, L, "bf16")
    q = torch.randn(1, 8, L, D, device="cuda").bfloat16()
    K, V = torch.randn(2, 1, 2, L, D, device="cuda").bfloat16().unbind(0)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.zeros(H.hata_prefill_workspace_size(d), dtype=torch.uint8, device="cuda")
    H.hata_prefill_attention(d, q, K, V, None, None, lens, 0.0, a, ws)
    H.hata_window_prefill(d, q, K, V, lens, L, 0, 0.0, b, ws)
    # |V| reaches about 5 where a row sees one or two keys: two roundings of each side, of values up to 5
    assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * 5


@pytest.mark.gpu
def test_too_long_is_clamped_and_flagged(H):
    d = H.dims_for(1, 2, 1, D, 128, 100, "bf16")
    q = torch.randn(1, 2, 100, D, device="cuda").bfloat16()
    K, V = torch.randn(2, 1, 1, 100, D, device="cuda").bfloat16().unbind(0)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    H.hata_window_prefill(d, q, K, V, torch.tensor([101], dtype=torch.int32, device="cuda"), 30, 2, 0.0, a, ws)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    H.hata_window_prefill(d, q, K, V, torch.tensor([100], dtype=torch.int32, device="cuda"), 30, 2, 0.0, b, ws)
    assert H.hata_read_device_status(ws) == 0 and torch.equal(a, b)
    H.hata_window_prefill(d, q, K, V, torch.tensor([-1], dtype=torch.int32, device="cuda"), 30, 2, 0.0, b, ws)
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["prefill", "tree"])
def test_a_wait_that_runs_out_is_reported(H, call):
    d = H.dims_for(2, 16, 2, D, 128, 600, "bf16", flags=H.HATA_FLAG_TEST_EXPIRE_WAIT)
    q = torch.randn(2, 16, 600, D, device="cuda").bfloat16()
    K, V = torch.randn(2, 2, 2, 600, D, device="cuda").bfloat16().unbind(0)
    lens = torch.tensor([600, 300], dtype=torch.int32, device="cuda")

    def run(flags):
        d.flags = flags
        if call == "prefill":
            out, ws = torch.zeros_like(q), torch.zeros(16, dtype=torch.uint8, device="cuda")
            H.hata_window_prefill(d, q, K, V, lens, 200, 4, 0.0, out, ws)
        else:
            qt = q[:, :, :40].contiguous()
            out = torch.zeros_like(qt)
            ws = torch.zeros(H.hata_span_workspace_size(d, 40), dtype=torch.uint8, device="cuda")
            H.hata_tree_attention(d, qt, K, V, lens, None, None, 0.0, out, ws)
        return H.hata_read_device_status(ws), out

    assert run(H.HATA_FLAG_TEST_EXPIRE_WAIT)[0] == H.HATA_ERR_TIMEOUT
    status, a = run(0)
    assert status == 0 and bool(a[0].any())
    assert torch.equal(run(0)[1], a)


def test_refusals(H):
    P = ctypes.c_void_p
    f, odd, null = P(0x1000), P(0x1008), P(0)
    d = H.dims_for(2, 4, 2, D, 128, 64, "bf16")

    def call(dd=d, q=f, K=f, V=f, lens=f, window=5, sink=0, scale=0.0, out=f, ws=f, wsb=16):
        return H.lib.hata_window_prefill(ctypes.byref(dd), q, K, V, lens, window, sink, scale, out, ws, wsb, null)

    assert call(dd=H.dims_for(2, 4, 2, D, 128, 64, "f32")) == 2
    assert call(q=null) == 1 and call(K=odd) == 1 and call(V=odd) == 1 and call(lens=null) == 1 and call(out=odd) == 1
    assert call(window=0) == 1 and call(sink=-1) == 1 and call(scale=float("inf")) == 1
    assert call(ws=null) == 5 and call(ws=odd) == 5 and call(wsb=8) == 5
