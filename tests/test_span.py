"""hata_window_decode and hata_tree_attention (contiguous and paged) against attention in 64 bits: lengths from one
to thousands, odd sizes, masks that leave rows empty, slots that nobody sees full of NaN, refusals."""
import ctypes

import pytest
import torch

from attention_testlib import attend, close

D = 128


@pytest.fixture(scope="module")
def H():
    import hash_aware_top_b200 as H

    return H


class Cache:
    def __init__(self, H, dtype, B, Hq, Hkv, max_seq, bs, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.bs, self.max_seq = H, bs, max_seq
        self.d = H.dims_for(B, Hq, Hkv, D, 128, max_seq, dtype)
        self.K = torch.randn(B, Hkv, max_seq, D, generator=g, device="cuda").to(dtype)
        self.V = torch.randn(B, Hkv, max_seq, D, generator=g, device="cuda").to(dtype)
        if bs:
            nb = -(-max_seq // bs)
            self.bt = torch.randperm(B * nb + 3, generator=g, device="cuda").int()[: B * nb].view(B, nb).contiguous()
        self.g = g

    def pools(self):
        """The same rows in pages; slots that no row fills are NaN."""
        B, Hkv, L, _ = self.K.shape
        nb, bs = self.bt.shape[1], self.bs
        out = []
        for t in (self.K, self.V):
            pad = torch.full((B, Hkv, nb * bs, D), float("nan"), device="cuda", dtype=t.dtype)
            pad[:, :, :L] = t
            pool = torch.full((B * nb + 3, Hkv, bs, D), float("nan"), device="cuda", dtype=t.dtype)
            pool[self.bt.long().flatten()] = pad.view(B, Hkv, nb, bs, D).transpose(1, 2).reshape(B * nb, Hkv, bs, D)
            out.append(pool)
        return out

    def workspace(self, n_tok=1):
        return torch.zeros(self.H.hata_span_workspace_size(self.d, n_tok), dtype=torch.uint8, device="cuda")


def window_case(H, dtype, B, Hq, Hkv, max_seq, bs, window, sink, lens, seed=0):
    c = Cache(H, dtype, B, Hq, Hkv, max_seq, bs, seed)
    q = torch.randn(B, Hq, D, generator=c.g, device="cuda").to(dtype)
    sees = torch.zeros(B, max_seq, dtype=torch.bool, device="cuda")
    at = torch.arange(max_seq, device="cuda")
    for b, L in enumerate(lens):
        sees[b] = (at < L) & ((at < sink) | (at >= L - window))
        c.K[b, :, ~sees[b]] = float("nan")  # nobody sees these
        c.V[b, :, ~sees[b]] = float("inf")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((B, Hq, D), 9.0, device="cuda", dtype=dtype)
    ws = c.workspace()
    for _ in range(2):  # the second call finds what the first one left in the workspace
        if bs:
            K, V = c.pools()
            H.hata_window_decode_paged(c.d, q, K, V, c.bt, bs, lens_d, window, sink, 0.0, out, ws)
        else:
            H.hata_window_decode(c.d, q, c.K, c.V, lens_d, window, sink, 0.0, out, ws)
        assert H.hata_read_device_status(ws) == 0
        G = Hq // Hkv
        for b, L in enumerate(lens):
            for g in range(Hkv):
                rows = slice(g * G, (g + 1) * G)
                want, absv, qk = attend(q[b, rows], c.K[b, g], c.V[b, g], sees[b][None].expand(G, max_seq))
                close(out[b, rows], want, absv, qk, min(L, window + sink), dtype)


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bs", [0, 16, 64, 256])
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (100, 4), (128, 128), (300, 0), (5000, 0), (77, 200), (2**31 - 1, 2**31 - 1)])
def test_window_decode(H, dtype, bs, window, sink):
    window_case(H, dtype, 4, 8, 2, 1111, bs, window, sink, [1111, 1, 500, 129], seed=window % 1000 + sink % 1000)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (12, 4), (32, 2), (7, 1)])
def test_window_decode_heads(H, dtype, Hq, Hkv):
    window_case(H, dtype, 3, Hq, Hkv, 260, 0, 130, 2, [260, 0, 17], seed=Hq)
    window_case(H, dtype, 1, Hq, Hkv, 9001, 32, 8000, 5, [9001], seed=Hq + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_window_decode_many_sequences(H, dtype):
    window_case(H, dtype, 70, 2, 1, 150, 16, 40, 3, [(37 * b) % 151 for b in range(70)])


@pytest.mark.gpu
def test_window_decode_clamps_and_flags(H):
    c = Cache(H, torch.bfloat16, 2, 4, 1, 64, 16, 0)
    q = torch.randn(2, 4, D, device="cuda").bfloat16()
    a, b = (torch.zeros(2, 4, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ws, (K, V) = c.workspace(), c.pools()
    lens = torch.tensor([99, -3], dtype=torch.int32, device="cuda")
    b.fill_(9.0)
    H.hata_window_decode(c.d, q, c.K, c.V, lens, 30, 2, 0.0, a, ws)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    H.hata_window_decode(c.d, q, c.K, c.V, lens.clamp(0, 64), 30, 2, 0.0, b, ws)
    assert torch.equal(a, b) and not bool(b[1].any())
    # a block outside the pool reads block 0
    bad, low = c.bt.clone(), c.bt.clone()
    bad[0, 3], low[0, 3] = 1000, 0
    K[torch.isnan(K)], V[torch.isnan(V)] = 0, 0
    lens = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
    H.hata_window_decode_paged(c.d, q, K, V, bad, 16, lens, 30, 2, 0.0, a, ws)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    H.hata_window_decode_paged(c.d, q, K, V, low, 16, lens, 30, 2, 0.0, b, ws)
    assert torch.equal(a, b) and H.hata_read_device_status(ws) == 0


def tree_case(H, dtype, B, T, Hq, Hkv, max_seq, bs, lens, n_new, mask="tree", seed=0):
    c = Cache(H, dtype, B, Hq, Hkv, max_seq, bs, seed)
    q = torch.randn(B, Hq, T, D, generator=c.g, device="cuda").to(dtype)
    among = torch.zeros(B, T, T, dtype=torch.bool, device="cuda")  # token i sees token j
    if mask is None:
        among[:] = torch.ones(T, T, device="cuda").tril().bool()
    elif mask == "tree":
        for b in range(B):
            for i in range(T):
                among[b, i, i] = True
                if i and i % 5:
                    among[b, i] |= among[b, (7 * i + b) % i]
    else:
        among[:] = torch.rand(B, T, T, generator=c.g, device="cuda") < mask
        among[:, ::3] = False  # rows that see no new token
    words = None
    if mask is not None:
        W = -(-T // 32)
        pad = torch.zeros(B, T, W * 32, dtype=torch.int64, device="cuda")
        pad[:, :, :T] = among
        words = (pad.view(B, T, W, 32) << torch.arange(32, device="cuda")).sum(-1)
        words = torch.where(words >= 2**31, words - 2**32, words).int().contiguous()
    at = torch.arange(max_seq, device="cuda")
    sees = torch.zeros(B, T, max_seq, dtype=torch.bool, device="cuda")
    for b, (L, n) in enumerate(zip(lens, n_new)):
        sees[b, :n] = at < L - n
        sees[b, :n, L - n:L] = among[b, :n, :n]
        seen = sees[b].any(0)
        c.K[b, :, ~seen], c.V[b, :, ~seen] = float("nan"), float("nan")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((B, Hq, T, D), 9.0, device="cuda", dtype=dtype)
    ws = c.workspace(T)
    args = (i32(lens), i32(n_new), words, 0.0, out, ws)
    if bs:
        H.hata_tree_attention_paged(c.d, q, *c.pools(), c.bt, bs, *args)
    else:
        H.hata_tree_attention(c.d, q, c.K, c.V, *args)
    assert H.hata_read_device_status(ws) == 0
    G = Hq // Hkv
    for b, (L, n) in enumerate(zip(lens, n_new)):
        for h in range(Hq):
            want, absv, qk = attend(q[b, h, :n], c.K[b, h // G], c.V[b, h // G], sees[b, :n])
            close(out[b, h, :n], want, absv, qk, max(L, 1), dtype)
    for b, n in enumerate(n_new):
        assert bool((out[b, :, n:] == 9.0).all())
    return c, q, words, out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bs", [0, 16, 256])
@pytest.mark.parametrize("T", [1, 2, 7, 9, 16, 31, 33, 64, 100, 128])
def test_tree(H, dtype, bs, T):
    tree_case(H, dtype, 3, T, 8, 2, 700, bs, [700, T, T + 131], [T, T, max(1, T - 1)], seed=T)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (16, 1), (12, 4)])
def test_tree_heads(H, dtype, Hq, Hkv):
    tree_case(H, dtype, 2, 13, Hq, Hkv, 3001, 64, [3001, 2999], [13, 9], seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [0, 16])
@pytest.mark.parametrize("T,max_seq", [(3, 5), (9, 9), (20, 130)])
def test_tree_caches_smaller_than_a_tile(H, bs, T, max_seq):
    tree_case(H, torch.bfloat16, 1, T, 16, 1, max_seq, bs, [max_seq], [T], seed=T)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hq", [(7, 4), (13, 4), (40, 4)])
def test_tree_many_sequences(H, dtype, T, Hq):
    """More sequences than a warp scans at a time, some without new tokens."""
    B = 45
    lens = [T + (61 * b) % 300 for b in range(B)]
    n_new = [0 if b % 7 == 3 else T - b % 3 for b in range(B)]
    tree_case(H, dtype, B, T, Hq, 1, 400, 16, lens, n_new, seed=B)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hq,Hkv", [(5, 4, 4), (40, 4, 1), (128, 8, 2)])
def test_tree_masks_that_leave_rows_empty(H, dtype, T, Hq, Hkv):
    tree_case(H, dtype, 3, T, Hq, Hkv, 400, 16, [T, T + 3, 0], [T, T, 0], mask=0.2, seed=T)
    tree_case(H, dtype, 3, T, Hq, Hkv, 400, 0, [T, 400, 130], [T, T, T if T < 130 else 130], mask=0.0, seed=T)


@pytest.mark.gpu
def test_tree_of_some_rows_over_a_long_cache(H):
    """Rows that a short cache gives to one kernel and a long one to the other."""
    tree_case(H, torch.bfloat16, 1, 12, 8, 2, 140000, 256, [139999], [12], seed=4)
    tree_case(H, torch.bfloat16, 1, 12, 8, 2, 4000, 256, [3999], [11], seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_chain(H, dtype):
    tree_case(H, dtype, 2, 50, 4, 2, 900, 64, [900, 50], [50, 50], mask=None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_tree_large_logits(H, dtype):
    """Queries thirty times as large: one key takes almost all of a row's weight, and maxima move often."""
    c = Cache(H, dtype, 1, 4, 1, 2000, 0, 3)
    q = (30 * torch.randn(1, 4, 9, D, generator=c.g, device="cuda")).to(dtype)
    out = torch.zeros_like(q)
    lens = torch.tensor([2000], dtype=torch.int32, device="cuda")
    H.hata_tree_attention(c.d, q, c.K, c.V, lens, None, None, 0.0, out, c.workspace(9))
    at = torch.arange(2000, device="cuda")
    sees = at[None] <= 1991 + torch.arange(9, device="cuda")[:, None]
    for h in range(4):
        want, absv, qk = attend(q[0, h], c.K[0, 0], c.V[0, 0], sees)
        close(out[0, h], want, absv, qk, 2000, dtype)


@pytest.mark.gpu
def test_tree_of_one_token_is_dense_decode(H):
    """A chain of one token computes what hata_dense_decode does, each within its own rounding (twice the bound)."""
    B, Hq, Hkv, L = 2, 8, 2, 3000
    c = Cache(H, torch.bfloat16, B, Hq, Hkv, L, 0, 1)
    q = torch.randn(B, Hq, 1, D, generator=c.g, device="cuda").bfloat16()
    lens = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    a, b = torch.zeros_like(q), torch.zeros(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros_like(b)
    H.hata_tree_attention(c.d, q, c.K, c.V, lens, None, None, 0.0, a, c.workspace())
    H.hata_window_decode(c.d, q[:, :, 0], c.K, c.V, lens, L, 0, 0.0, w, c.workspace())
    ws = torch.zeros(H.hata_dense_workspace_size(c.d), dtype=torch.uint8, device="cuda")
    H.hata_dense_decode(c.d, q[:, :, 0].contiguous(), c.K, c.V, lens, 0.0, b, ws)
    # p and the output are rounded by each: 4 half steps of values that sum p |v| < 4 bounds
    assert float((a[:, :, 0].float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * 4
    assert float((w.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * 4


@pytest.mark.gpu
def test_tree_bad_lengths_are_flagged_and_left(H):
    c = Cache(H, torch.bfloat16, 4, 2, 1, 64, 0, 0)
    q = torch.randn(4, 2, 5, D, device="cuda").bfloat16()
    out = torch.full_like(q, 9.0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = c.workspace(5)
    H.hata_tree_attention(c.d, q, c.K, c.V, i32([65, 4, 20, 20]), i32([5, 5, 6, 5]), None, 0.0, out, ws)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    assert bool((out[:3] == 9.0).all()) and not bool((out[3] == 9.0).all(-1).any())


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq", [(1, 4), (6, 4), (40, 4)])
def test_offsets_past_32_bits(H, T, Hq):
    """Pages at the end of pools of more than 2^31 elements, and slots at the end of such a contiguous cache."""
    B, Hkv, bs = 1, 1, 256
    n = 2**31 // (Hkv * bs * D) + 600
    K, V = (torch.empty(n, Hkv, bs, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    L = 1000
    d = H.dims_for(B, Hq, Hkv, D, 128, L, "bf16")
    bt = torch.tensor([[n - 1, n - 3, n - 599, n - 2]], dtype=torch.int32, device="cuda")
    q = torch.randn(B, Hq, T, D, device="cuda").bfloat16()
    Kd, Vd = torch.randn(2, L, D, device="cuda").bfloat16().unbind(0)
    for i in range(4):
        K[bt[0, i].long(), 0, : min(bs, L - i * bs)] = Kd[i * bs:(i + 1) * bs]
        V[bt[0, i].long(), 0, : min(bs, L - i * bs)] = Vd[i * bs:(i + 1) * bs]
    out, ws = torch.zeros_like(q), torch.zeros(H.hata_span_workspace_size(d, T), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    H.hata_tree_attention_paged(d, q, K, V, bt, bs, lens, None, None, 0.0, out, ws)
    sees = torch.arange(L, device="cuda")[None] <= L - T + torch.arange(T, device="cuda")[:, None]
    for h in range(Hq):
        want, absv, qk = attend(q[0, h], Kd, Vd, sees)
        close(out[0, h], want, absv, qk, L, torch.bfloat16)
    # the same memory as one contiguous cache of 2^24 slots and more
    S = n * bs
    K, V = K.view(1, 1, S, D), V.view(1, 1, S, D)
    K[0, 0, S - L:], V[0, 0, S - L:] = Kd, Vd
    K[0, 0, :5], V[0, 0, :5] = Kd[:5], Vd[:5]
    d = H.dims_for(B, Hq, Hkv, D, 128, S, "bf16")
    lens = torch.tensor([S], dtype=torch.int32, device="cuda")
    out = torch.zeros(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(H.hata_span_workspace_size(d, 1), dtype=torch.uint8, device="cuda")
    H.hata_window_decode(d, q[:, :, 0].contiguous(), K, V, lens, L, 5, 0.0, out, ws)
    for h in range(Hq):
        want, absv, qk = attend(q[0, h, :1], torch.cat([Kd[:5], Kd]), torch.cat([Vd[:5], Vd]), torch.ones(1, L + 5, dtype=torch.bool, device="cuda"))
        close(out[0, h][None], want, absv, qk, L + 5, torch.bfloat16)
    x = torch.randn(1, T, Hq + 2, D, device="cuda").bfloat16()
    q_out = torch.zeros(1, Hq, T, D, device="cuda", dtype=torch.bfloat16)
    H.hata_norm_rope(d, x[:, :, :Hq], x[:, :, Hq:Hq + 1], x[:, :, Hq + 1:], None, None, 1e-6, None, False, None, None, lens, q_out, K, V, ws)
    assert torch.equal(K[0, 0, S - T:], x[0, :, Hq]) and torch.equal(V[0, 0, S - T:], x[0, :, Hq + 1])
    keep = torch.arange(T, dtype=torch.int32, device="cuda")[None].contiguous()
    keep[0, 0] = T - 1
    H.hata_compact_kv(d, keep, torch.ones(1, dtype=torch.int32, device="cuda"), None, lens, K, V, None, None, ws)
    assert torch.equal(K[0, 0, S - T], x[0, T - 1, Hq]) and H.hata_read_device_status(ws) == 0


@pytest.mark.gpu
def test_captured_and_replayed(H):
    """A captured window decode and tree attention give the eager results, replayed with other inputs."""
    c = Cache(H, torch.bfloat16, 2, 8, 2, 500, 16, 5)
    K, V = c.pools()
    K[torch.isnan(K)], V[torch.isnan(V)] = 0, 0
    q = torch.randn(2, 8, 6, D, device="cuda").bfloat16()
    q1 = q[:, :, 0].contiguous()
    lens = torch.tensor([500, 300], dtype=torch.int32, device="cuda")
    out, out1 = torch.zeros_like(q), torch.zeros_like(q1)
    ws, ws1 = c.workspace(6), c.workspace()

    def both():
        H.hata_tree_attention_paged(c.d, q, K, V, c.bt, 16, lens, None, None, 0.0, out, ws)
        H.hata_window_decode_paged(c.d, q1, K, V, c.bt, 16, lens, 100, 4, 0.0, out1, ws1)

    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for seed in range(3):
        q.copy_(torch.randn(2, 8, 6, D, device="cuda"))
        q1.copy_(q[:, :, 1])
        lens.copy_(torch.tensor([400 - 7 * seed, 77 + seed]))
        both()
        torch.cuda.synchronize()
        want, want1 = out.clone(), out1.clone()
        out.zero_(), out1.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out1, want1)


@pytest.mark.gpu
def test_binding_refuses(H):
    c = Cache(H, torch.bfloat16, 2, 4, 2, 64, 0, 0)
    q = torch.zeros(2, 4, 3, D, device="cuda", dtype=torch.bfloat16)
    lens, ws = torch.ones(2, dtype=torch.int32, device="cuda"), c.workspace(3)
    with pytest.raises(ValueError, match="shape"):
        H.hata_tree_attention(c.d, q, c.K, c.V, lens, None, torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda"), 0.0, q.clone(), ws)
    with pytest.raises(ValueError, match="contiguous"):
        H.hata_tree_attention(c.d, q.transpose(1, 2).contiguous().transpose(1, 2), c.K, c.V, lens, None, None, 0.0,
                              q.clone(), ws)
    with pytest.raises(TypeError, match="bfloat16"):
        H.hata_tree_attention(c.d, q.float(), c.K, c.V, lens, None, None, 0.0, q.clone(), ws)
    with pytest.raises(H.HataError, match="workspace"):
        H.hata_tree_attention(c.d, q, c.K, c.V, lens, None, None, 0.0, q.clone(), ws[:256])
    with pytest.raises(H.HataError, match="invalid"):
        H.hata_window_decode(c.d, q[:, :, 0].contiguous(), c.K, c.V, lens, 0, 0, 0.0, q[:, :, 0].contiguous(), ws)


def test_refusals(H):
    P = ctypes.c_void_p
    f, odd, null = P(0x1000), P(0x1008), P(0)
    d = H.dims_for(2, 4, 2, D, 128, 64, "bf16")
    n = ctypes.c_size_t(0)
    assert H.lib.hata_span_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)) == 1
    assert H.lib.hata_span_workspace_size(ctypes.byref(d), 129, ctypes.byref(n)) == 2
    assert H.lib.hata_span_workspace_size(ctypes.byref(d), 128, ctypes.byref(n)) == 0 and n.value > 0

    def win(q=f, K=f, lens=f, window=4, sink=0, scale=0.0, out=f, ws=f, wsb=1 << 40):
        return H.lib.hata_window_decode(ctypes.byref(d), q, K, f, lens, window, sink, scale, out, ws, wsb, null)

    assert win(q=null) == 1 and win(K=odd) == 1 and win(lens=null) == 1 and win(out=null) == 1
    assert win(window=0) == 1 and win(window=-1) == 1 and win(sink=-1) == 1 and win(scale=float("nan")) == 1
    assert win(scale=float("inf")) == 1 and win(ws=null) == 5 and win(ws=odd) == 5 and win(wsb=64) == 5

    def tree(T=4, q=f, mask=null, wsb=1 << 40, ws=f):
        return H.lib.hata_tree_attention(ctypes.byref(d), T, q, f, f, f, null, mask, 0.0, f, ws, wsb, null)

    assert tree(T=0) == 1 and tree(T=129) == 2 and tree(q=odd) == 1 and tree(mask=P(0x1002)) == 1
    assert tree(wsb=64) == 5 and tree(ws=null) == 5
    assert H.lib.hata_tree_attention_paged(ctypes.byref(d), 4, f, f, f, f, 12, 4, f, null, null, 0.0, f, f, 1 << 40, null) == 1
    assert H.lib.hata_window_decode_paged(ctypes.byref(d), f, f, f, null, 16, 4, f, 4, 0, 0.0, f, f, 1 << 40, null) == 1


def test_group_sizes(H):
    """Up to 16 query heads for a KV head, in every call; more are unsupported."""
    P = ctypes.c_void_p
    f, null, n = P(0x1000), P(0), ctypes.c_size_t(0)
    for G, status in ((16, 0), (17, 2), (32, 2)):
        d = ctypes.byref(H.dims_for(1, 2 * G, 2, D, 128, 64, "bf16"))
        assert H.lib.hata_span_workspace_size(d, 4, ctypes.byref(n)) == status
        assert H.lib.hata_pages_workspace_size(d, ctypes.byref(n)) == status
        # a bad argument where the group is allowed, so that nothing is launched
        assert H.lib.hata_window_decode(d, null, f, f, f, 4, 0, 0.0, f, f, 1 << 40, null) == (status or 1)
        assert H.lib.hata_window_prefill(d, null, f, f, f, 4, 0, 0.0, f, f, 16, null) == (status or 1)
        assert H.lib.hata_tree_attention(d, 4, null, f, f, f, null, null, 0.0, f, f, 1 << 40, null) == (status or 1)
        assert H.lib.hata_norm_rope(d, 1, null, 4096, f, 256, f, 256, null, null, 1e-6, f, 64, 128, 0, null, null, f, f, f, f, f, 16,
                                    null) == (status or 1)
        assert H.lib.hata_compact_kv(d, 4, null, f, null, f, f, f, null, null, f, 16, null) == (status or 1)
