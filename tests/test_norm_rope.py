"""hata_norm_rope: norms of queries and keys for each head, position rotation and cache append in one pass,
contiguous and paged, against the formula in 64 bits; the table; refusals."""
import ctypes

import pytest
import torch

D = 128
EPS = 1e-6


@pytest.fixture(scope="module")
def H():
    import hash_aware_top_b200 as H

    return H


def rounding(dtype):
    """Half a step of the type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def reference(x, w, table, pos, inter):
    """x [..., D] and pos [...] (int64) -> value in 64 bits and the magnitude that rounding errors scale with."""
    x = x.double()
    y = x if w is None else x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    mag = y.abs()
    if table is None:
        return y, mag
    half = table.shape[2]
    cos, sin = table[pos, 0].double(), table[pos, 1].double()
    out, m = y.clone(), mag.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        ya, yb, c, s = y[..., a], y[..., b], cos[..., i], sin[..., i]
        out[..., a], out[..., b] = ya * c - yb * s, yb * c + ya * s
        m[..., a] = ya.abs() * c.abs() + yb.abs() * s.abs()
        m[..., b] = yb.abs() * c.abs() + ya.abs() * s.abs()
    return out, m


def close(got, want, mag, dtype):
    """fp32 arithmetic: the mean square of 128 terms is off by at most 130 half steps, so its root by 65 (and the
    reciprocal root by 4 more), two products, and three roundings of a rotation: under 80 half steps of fp32 of
    the magnitude; then one rounding to the type."""
    err = (got.double() - want).abs()
    tol = 80 * rounding(torch.float32) * mag + (rounding(dtype) * want.abs() if dtype != torch.float32 else 0) * 1.01
    assert bool((err <= tol + 1e-30).all()), float((err - tol).max())


def make(H, dtype, B, T, Hq, Hkv, max_seq, rot, inter, seed, fused=True, pos=False, ragged=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if fused:
        x = r(B, T, Hq + 2 * Hkv, D).to(dtype)
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    else:
        q, k, v = r(B, T, Hq, D).to(dtype), r(B, T, Hkv, D).to(dtype), r(B, T, Hkv, D).to(dtype)
    table = H.hata_rope_table(max_seq + 7, rot, 10000.0) if rot else None
    n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    nn = n if ragged else torch.full((B,), T, dtype=torch.int32, device="cuda")
    lens = (nn + (torch.rand(B, generator=g, device="cuda") * (max_seq - nn + 1)).int()).clamp(max=max_seq).int()
    positions = torch.randint(0, max_seq + 7, (B, T), generator=g, device="cuda", dtype=torch.int32) if pos else None
    return dict(q=q, k=k, v=v, wq=1 + 0.3 * r(D), wk=1 + 0.3 * r(D), table=table, n=n, nn=nn, lens=lens, positions=positions)


def check(H, dtype, B, T, Hq, Hkv, max_seq, rot, inter, bs, seed=0, weights=True, **kw):
    m = make(H, dtype, B, T, Hq, Hkv, max_seq, rot, inter, seed, **kw)
    d = H.dims_for(B, Hq, Hkv, D, 128, max_seq, dtype)
    wq, wk = (m["wq"], m["wk"]) if weights else (None, None)
    q_out = torch.full((B, Hq, T, D), 7.0, device="cuda", dtype=dtype)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    args = (d, m["q"], m["k"], m["v"], wq, wk, EPS, m["table"], inter, m["n"], m["positions"], m["lens"], q_out)
    if bs:
        nb = -(-max_seq // bs)
        bt = torch.randperm(B * nb + 2, device="cuda").int()[: B * nb].view(B, nb).contiguous()
        K = torch.full((B * nb + 2, Hkv, bs, D), 5.0, device="cuda", dtype=dtype)
        V = K.clone()
        H.hata_norm_rope_paged(*args, K, V, bt, bs, ws)
    else:
        K = torch.full((B, Hkv, max_seq, D), 5.0, device="cuda", dtype=dtype)
        V = K.clone()
        H.hata_norm_rope(*args, K, V, ws)
    assert H.hata_read_device_status(ws) == 0
    wantK, wantV = K.clone(), V.clone()
    for b in range(B):
        n, L = int(m["nn"][b]), int(m["lens"][b])
        slot = torch.arange(L - n, L, device="cuda")
        pos = slot if m["positions"] is None else m["positions"][b, :n].long()
        want, mag = reference(m["q"][b, :n], wq, m["table"], pos[:, None].expand(n, Hq), inter)
        close(q_out[b, :, :n].transpose(0, 1), want, mag, dtype)
        assert bool((q_out[b, :, n:] == 7.0).all())
        want, mag = reference(m["k"][b, :n], wk, m["table"], pos[:, None].expand(n, Hkv), inter)
        if bs:
            page, off = bt[b].long()[slot // bs], slot % bs
            close(K[page, :, off], want, mag, dtype)
            assert torch.equal(V[page, :, off], m["v"][b, :n])
            wantK[page, :, off], wantV[page, :, off] = 5.0, 5.0
        else:
            close(K[b, :, L - n:L].transpose(0, 1), want, mag, dtype)
            assert torch.equal(V[b, :, L - n:L].transpose(0, 1), m["v"][b, :n])
            wantK[b, :, L - n:L], wantV[b, :, L - n:L] = 5.0, 5.0
    # every other cache row is as it was
    assert bool((wantK == 5.0).all()) and bool((wantV == 5.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 96, 32, 16, 0])
def test_rotations(H, dtype, inter, rot):
    check(H, dtype, 3, 5, 6, 2, 40, rot, inter, 0, seed=rot)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,Hkv,max_seq,bs", [
    (1, 1, 1, 1, 1, 0), (1, 1, 1, 1, 16, 16), (16, 1, 32, 8, 300, 64), (2, 37, 5, 5, 64, 16), (5, 9, 16, 1, 33, 16),
    (2, 130, 12, 4, 131, 0), (3, 8, 7, 7, 300, 256),
])
def test_shapes(H, dtype, B, T, Hq, Hkv, max_seq, bs):
    check(H, dtype, B, T, Hq, Hkv, max_seq, 64, False, bs, seed=T)
    check(H, dtype, B, T, Hq, Hkv, max_seq, 128, True, bs, seed=T + 1, fused=False, pos=True, ragged=False)


@pytest.mark.gpu
def test_no_norm(H):
    check(H, torch.bfloat16, 2, 3, 4, 2, 32, 128, False, 0, weights=False)
    check(H, torch.float32, 2, 3, 4, 2, 32, 0, False, 16, weights=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 32, 96])
def test_elements_that_do_not_turn_are_copies_without_a_weight(H, dtype, inter, rot):
    """Infinities, NaN, zeros of both signs and their neighbours: y = x for every element past rot_dim, bit for bit."""
    B, T, Hq, Hkv, L = 1, 2, 3, 1, 8
    d = H.dims_for(B, Hq, Hkv, D, 128, L, dtype)
    g = torch.Generator(device="cuda").manual_seed(rot)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(dtype)
    x[..., 100], x[..., 103], x[..., 106], x[..., 127] = float("inf"), float("-inf"), float("nan"), -0.0
    q_out = torch.zeros(B, Hq, T, D, device="cuda", dtype=dtype)
    K, V = torch.zeros(2, B, Hkv, L, D, device="cuda", dtype=dtype).unbind(0)
    lens, ws = torch.tensor([5], dtype=torch.int32, device="cuda"), torch.zeros(16, dtype=torch.uint8, device="cuda")
    table = H.hata_rope_table(L, rot, 1e4) if rot else None
    H.hata_norm_rope(d, x[:, :, :Hq], x[:, :, Hq:Hq + 1], x[:, :, Hq + 1:], None, None, EPS, table, inter, None, None, lens,
                     q_out, K, V, ws)
    assert H.hata_read_device_status(ws) == 0
    bits = lambda t: t.contiguous().view(torch.int32 if dtype == torch.float32 else torch.int16)  # noqa: E731
    nan = torch.isnan(x)
    for got, want, n in ((q_out[0].transpose(0, 1), x[0, :, :Hq], nan[0, :, :Hq]),
                         (K[0, :, 3:5].transpose(0, 1), x[0, :, Hq:Hq + 1], nan[0, :, Hq:Hq + 1])):
        assert torch.equal(torch.isnan(got), n)
        assert torch.equal(bits(got[..., rot:])[~n[..., rot:]], bits(want[..., rot:])[~n[..., rot:]])
    # with a weight, elements that do not turn are x r w of their own x alone
    x[..., 100], x[..., 103], x[..., 106] = 1e18, -1e18, 0.0
    w = torch.ones(D, device="cuda")
    w[102] = float("inf")  # the weight of an interleaved neighbour
    H.hata_norm_rope(d, x[:, :, :Hq], x[:, :, Hq:Hq + 1], x[:, :, Hq + 1:], w, w, EPS, table, inter, None, None, lens, q_out, K, V, ws)
    assert bool(torch.isfinite(q_out[..., 103]).all()) and bool(torch.isfinite(K[0, :, 3:5, 103]).all())


@pytest.mark.gpu
def test_table(H):
    """Angles in 64 bits, rounded once: half a step of fp32 of values up to 1, and as much again for the 64-bit
    functions' last places at far positions (t = 2e5 has angles of 2e5 * 2^-53)."""
    t = H.hata_rope_table(200001, 32, 500000.0)
    pos = torch.tensor([0, 1, 17, 131071, 200000])
    ang = pos[:, None].double() * 500000.0 ** (-torch.arange(16).double() / 16)
    got = t[pos.cuda()].cpu().double()
    tol = rounding(torch.float32) * 1.01 + 2e5 * 2.0 ** -50
    assert float((got[:, 0] - ang.cos()).abs().max()) <= tol and float((got[:, 1] - ang.sin()).abs().max()) <= tol


@pytest.mark.gpu
def test_replaces_the_append_before_a_decode_step(H):
    """One new token per sequence without norms and rotation is what hata_append_kv writes."""
    B, Hq, Hkv, L = 3, 8, 2, 50
    d = H.dims_for(B, Hq, Hkv, D, 128, L, "bf16")
    x = torch.randn(B, 1, Hq + 2 * Hkv, D, device="cuda").bfloat16()
    lens = torch.tensor([1, 50, 20], dtype=torch.int32, device="cuda")
    K1, V1 = torch.zeros(2, B, Hkv, L, D, device="cuda", dtype=torch.bfloat16).unbind(0)
    K2, V2 = K1.clone(), V1.clone()
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    q_out = torch.empty(B, Hq, 1, D, device="cuda", dtype=torch.bfloat16)
    H.hata_norm_rope(d, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], None, None, EPS, None, False, None, None,
                     lens, q_out, K1, V1, ws)
    H.hata_append_kv(d, x[:, 0, Hq:Hq + Hkv].contiguous(), x[:, 0, Hq + Hkv:].contiguous(), K2, V2, lens)
    assert torch.equal(K1, K2) and torch.equal(V1, V2) and torch.equal(q_out[:, :, 0], x[:, 0, :Hq])


@pytest.mark.gpu
def test_bad_lengths_positions_and_blocks_are_flagged_and_left(H):
    B, T, Hq, Hkv, L, bs = 4, 3, 2, 1, 32, 16
    d = H.dims_for(B, Hq, Hkv, D, 128, L, "bf16")
    x = torch.randn(B, T, Hq + 2 * Hkv, D, device="cuda").bfloat16()
    table = H.hata_rope_table(20, 128, 1e4)
    lens = torch.tensor([2, 33, 10, 10], dtype=torch.int32, device="cuda")  # shorter than its new tokens; too long
    n = torch.tensor([3, 3, 4, 3], dtype=torch.int32, device="cuda")  # the third has more than T
    q_out = torch.full((B, Hq, T, D), 7.0, device="cuda", dtype=torch.bfloat16)
    K = torch.full((8, Hkv, bs, D), 5.0, device="cuda", dtype=torch.bfloat16)
    V, ws = K.clone(), torch.zeros(16, dtype=torch.uint8, device="cuda")
    bt = torch.arange(8, dtype=torch.int32, device="cuda").view(B, 2).contiguous()
    call = lambda pos, bt: H.hata_norm_rope_paged(  # noqa: E731
        d, x[:, :, :2], x[:, :, 2:3], x[:, :, 3:], None, None, EPS, table, False, n, pos, lens, q_out, K, V, bt, bs, ws)
    call(None, bt)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    assert bool((q_out[:3] == 7.0).all()) and bool((K[:6] == 5.0).all()) and not bool((q_out[3] == 7.0).any())
    # a position outside the table: that token alone
    lens.fill_(16), n.fill_(3)
    pos = torch.tensor([[0, 20, 1], [0, -1, 1], [0, 1, 2], [0, 1, 2]], dtype=torch.int32, device="cuda")
    q_out.fill_(7.0)
    call(pos, bt)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    assert bool((q_out[:2, :, 1] == 7.0).all()) and not bool((q_out[:2, :, [0, 2]] == 7.0).all(-1).any())
    # a block outside the pool: its rows alone
    K.fill_(5.0), q_out.fill_(7.0)
    bad = bt.clone()
    bad[0, 0], bad[1, 0] = 8, -1
    call(None, bad)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    assert bool((K[:4] == 5.0).all()) and not bool((K[4, :, 13:] == 5.0).all()) and not bool((q_out == 7.0).all(-1).any())


def test_refusals(H):
    P = ctypes.c_void_p
    f, odd, null = P(0x1000), P(0x1008), P(0)
    d = H.dims_for(2, 4, 2, D, 128, 64, "bf16")

    def call(dd=d, n_tok=3, q=f, qs=512, ks=256, vs=256, eps=EPS, table=f, n_pos=64, rot=128, lens=f, out=f, K=f, ws=f, wsb=16):
        return H.lib.hata_norm_rope(ctypes.byref(dd), n_tok, q, qs, f, ks, f, vs, null, null, eps, table, n_pos, rot, 0,
                                    null, null, lens, out, K, f, ws, wsb, null)

    assert call(q=null) == 1 and call(q=odd) == 1 and call(out=odd) == 1 and call(K=null) == 1 and call(lens=null) == 1
    assert call(n_tok=0) == 1 and call(qs=511) == 1 and call(qs=504) == 1 and call(ks=260) == 1 and call(vs=128) == 1
    assert call(eps=0.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(rot=130) == 1 and call(rot=-2) == 1 and call(rot=7) == 1 and call(rot=20) == 2
    assert call(table=null) == 1 and call(n_pos=0) == 1 and call(ws=null) == 5 and call(ws=odd) == 5 and call(wsb=8) == 5
    assert call(dd=H.dims_for(2, 4, 2, 64, 128, 64, "bf16")) == 2
    paged = lambda bt, bs, n: H.lib.hata_norm_rope_paged(  # noqa: E731
        ctypes.byref(d), 3, f, 512, f, 256, f, 256, null, null, EPS, f, 64, 128, 0, null, null, f, f, f, f, bt, bs, n, f, 16,
        null)
    assert paged(null, 16, 4) == 1 and paged(f, 24, 4) == 1 and paged(f, 8, 4) == 1 and paged(f, 16, 0) == 1
    assert H.lib.hata_rope_table(f, 0, 64, 1e4, null) == 1 and H.lib.hata_rope_table(f, 4, 20, 1e4, null) == 2
    assert H.lib.hata_rope_table(null, 4, 64, 1e4, null) == 1 and H.lib.hata_rope_table(f, 4, 64, -1.0, null) == 1


def test_binding_refuses_cpu_tensors(H):
    d = H.dims_for(1, 2, 1, D, 128, 16, "f32")
    x = torch.zeros(1, 1, 4, D)
    with pytest.raises(ValueError, match="CUDA tensor"):
        H.hata_norm_rope(d, x[:, :, :2], x[:, :, 2:3], x[:, :, 3:], None, None, EPS, None, False, None, None,
                         torch.ones(1, dtype=torch.int32), x, x, x, torch.zeros(16, dtype=torch.uint8))


@pytest.mark.gpu
def test_binding_refuses_layouts(H):
    d = H.dims_for(2, 4, 2, D, 128, 16, "f32")
    x = torch.zeros(2, 3, 8, D, device="cuda")
    lens = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    out, K = torch.zeros(2, 4, 3, D, device="cuda"), torch.zeros(2, 2, 16, D, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    call = lambda q, k: H.hata_norm_rope(d, q, k, x[:, :, 6:], None, None, EPS, None, False, None, None, lens, out, K, K.clone(), ws)  # noqa: E731
    with pytest.raises(ValueError, match="side by side"):
        call(x[:, :, ::2], x[:, :, 4:6])  # every other head
    with pytest.raises(ValueError, match="side by side"):
        call(torch.zeros(3, 2, 4, D, device="cuda").transpose(0, 1), x[:, :, 4:6])  # sequences inside tokens
    with pytest.raises(TypeError, match="float32"):
        call(x[:, :, :4].bfloat16(), x[:, :, 4:6])
    with pytest.raises(ValueError, match="shape"):
        call(x[:, :, :4], x[:, :, 4:7])
