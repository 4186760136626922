"""The serving operators beside the decode step, as measured: what each case is, its inputs, one pass through the
operator (plain torch operations, or the framework's calls where `own` is true), its work, and its exact value.

Operators:
  norm_rope  norms of queries and keys for each head, position rotation, and the cache append, in one pass
  window     attention with a sliding window and a few first tokens that stay visible: decode and prefill
  tree       attention of a tree of drafted tokens over a cache
  pages      a paged cache's bookkeeping: fork, copy on write, allocate and free
  compact    accepted rows of a cache moved to the front of the drafted ones
"""
import math

import torch

own = False

D = 128


def listed():
    return [
        # one decode step of 16 sequences writing their new token into a paged cache: latency
        dict(name="norm_rope_decode_b16_paged", op="norm_rope", dtype="bf16", B=16, T=1, Hq=32, Hkv=8, max_seq=4096, bs=64,
             rot=128, inter=False, ragged=True, positions=False),
        # the projections of four long prompts of different lengths
        dict(name="norm_rope_prefill_b4_8k", op="norm_rope", dtype="bf16", B=4, T=8192, Hq=32, Hkv=8, max_seq=8192, bs=0,
             rot=128, inter=False, ragged=True, positions=False),
        # a small tree of drafted tokens, rotated by depth, interleaved pairs, half of each head rotated
        dict(name="norm_rope_tree_f32", op="norm_rope", dtype="f32", B=2, T=13, Hq=8, Hkv=2, max_seq=1024, bs=0,
             rot=64, inter=True, ragged=False, positions=True),
        # one decode step of a single long conversation in a sliding-window layer
        dict(name="window_decode_b1_128k", op="window_decode", dtype="bf16", B=1, Hq=32, Hkv=8, max_seq=131072, bs=0,
             window=4096, sink=4),
        # a batch of ragged conversations over a paged cache
        dict(name="window_decode_b16_paged", op="window_decode", dtype="bf16", B=16, Hq=32, Hkv=8, max_seq=16384, bs=64,
             window=8191, sink=16),
        # one long prompt through a sliding-window layer
        dict(name="window_prefill_b1_8k", op="window_prefill", dtype="bf16", B=1, Hq=32, Hkv=8, L=8192, window=1024,
             sink=4, ragged=False),
        # short prompts of odd lengths, a window that ends inside a tile, sinks longer than a tile
        dict(name="window_prefill_b3_odd", op="window_prefill", dtype="bf16", B=3, Hq=8, Hkv=2, L=2049, window=333,
             sink=130, ragged=True),
        # a few drafted tokens of one conversation over a paged cache: latency and bandwidth
        dict(name="tree_b1_7_32k_paged", op="tree", dtype="bf16", B=1, T=7, Hq=32, Hkv=8, L=32768, bs=64, ragged=False),
        # wide trees of four conversations at long context
        dict(name="tree_b4_64_64k", op="tree", dtype="bf16", B=4, T=64, Hq=32, Hkv=8, L=65536, bs=0, ragged=True),
        # single precision, one head for each cache head
        dict(name="tree_f32_4k", op="tree", dtype="f32", B=1, T=13, Hq=4, Hkv=4, L=4096, bs=0, ragged=False),
        # a beam step: roll back, fork eight sequences into 24 more, grow all by a few tokens
        dict(name="pages_fork_32", op="pages", dtype="bf16", parents=8, forks=3, Hkv=8, max_seq=16384, bs=64, r=128,
             grow=5, spare=256),
        # the accepted path of a tree of 64 nodes, 16 sequences
        dict(name="compact_b16_paged", op="compact", dtype="bf16", B=16, T=64, Hkv=8, max_seq=8192, bs=64, r=128, most=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "window_decode", "window_prefill", "tree", "pages", "compact"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    Hq, Hkv = rng.choice([(32, 8), (8, 2), (4, 4), (1, 1), (16, 2), (12, 4), (16, 1)])
    bs = rng.choice([0, 16, 64, 256])
    if op == "norm_rope":
        B = _log(rng, 1, 32)
        T = _log(rng, 1, min(8192, 32768 // B))
        return dict(op=op, dtype=dtype, B=B, T=T, Hq=Hq, Hkv=Hkv, max_seq=T + _log(rng, 1, 2000), bs=bs,
                    rot=rng.choice([128, 128, 96, 64, 32]), inter=rng.random() < 0.5, ragged=rng.random() < 0.5,
                    positions=rng.random() < 0.5)
    if op == "window_decode":
        B = _log(rng, 1, 16)
        max_seq = _log(rng, 64, 131072 // B)
        return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, max_seq=max_seq, bs=bs, window=_log(rng, 1, 8192),
                    sink=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
    if op == "window_prefill":
        B = _log(rng, 1, 4)
        return dict(op=op, dtype="bf16", B=B, Hq=Hq, Hkv=Hkv, L=_log(rng, 1, int(8192 / math.sqrt(B))),
                    window=_log(rng, 1, 8192), sink=rng.choice([0, 1, 4, _log(rng, 1, 300)]), ragged=rng.random() < 0.5)
    if op == "tree":
        B, T = _log(rng, 1, 4), _log(rng, 1, 64)
        L = T + _log(rng, 1, (8192 if dtype == "f32" else 65000) // B)
        return dict(op=op, dtype=dtype, B=B, T=T, Hq=Hq, Hkv=Hkv, L=L, bs=bs, ragged=rng.random() < 0.5)
    bs = bs or 64
    if op == "pages":
        return dict(op=op, dtype=dtype, parents=_log(rng, 1, 8), forks=rng.randint(1, 4), Hkv=Hkv,
                    max_seq=_log(rng, 200, 8192), bs=bs, r=rng.choice([32, 128]), grow=_log(rng, 1, 100),
                    spare=rng.randint(0, 300))
    return dict(op=op, dtype=dtype, B=_log(rng, 1, 32), T=rng.randint(9, 128), Hkv=Hkv, max_seq=_log(rng, 200, 8192), bs=bs,
                r=rng.choice([32, 128]), most=rng.randint(1, 9))


# ---------------------------------------------------------------- inputs


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _table(g, B, max_blocks, spare):
    """A block table of distinct, scattered pages, and the number of pages of the pool."""
    n = B * max_blocks + spare
    perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    return perm[: B * max_blocks].reshape(B, max_blocks).contiguous(), n


def _cache(case, g, B, Hkv, max_seq, bs):
    """K and V, contiguous or as pools of pages with a block table."""
    t = _type(case)
    if not bs:
        shape, bt = (B, Hkv, max_seq, D), None
    else:
        bt, n = _table(g, B, -(-max_seq // bs), 3)
        shape = (n, Hkv, bs, D)
    return (torch.randn(shape, generator=g, device="cuda", dtype=t), torch.randn(shape, generator=g, device="cuda", dtype=t), bt)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _parents(g, B, T):
    """A random tree for each sequence: the parent of node i is an earlier node, or -1 for the first level."""
    u = torch.rand((B, T), generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    return (torch.floor(u * (i + 1)).to(torch.int64) - 1).clamp(max=T - 2)


def _ancestors(parent):
    """[B][T][T] truth values: node i sees node j (its ancestors and itself), and each node's depth."""
    B, T = parent.shape
    sees = torch.eye(T, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    at = parent.clone()
    b = torch.arange(B, device="cuda")[:, None].expand(B, T)
    i = torch.arange(T, device="cuda")[None].expand(B, T)
    for _ in range(T):
        ok = at >= 0
        if not bool(ok.any()):
            break
        sees[b[ok], i[ok], at[ok]] = True
        at = torch.where(ok, torch.gather(parent, 1, at.clamp(min=0)), at)
    return sees, sees.sum(-1) - 1


def _bits(sees):
    """The tree mask as words: bit j of row i is set where node i sees node j."""
    B, T, _ = sees.shape
    W = -(-T // 32)
    pad = torch.zeros((B, T, W * 32), dtype=torch.int64, device="cuda")
    pad[:, :, :T] = sees
    words = (pad.view(B, T, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 2**31, words - 2**32, words).to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, op = _type(case), case["op"]
    s = dict(case=case)
    s["ws"] = torch.zeros(96 << 20, dtype=torch.uint8, device="cuda")
    if op == "norm_rope":
        B, T, Hq, Hkv, max_seq, rot = (case[k] for k in ("B", "T", "Hq", "Hkv", "max_seq", "rot"))
        # one projection's output: the heads of q, k and v side by side for each token
        qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=g, device="cuda", dtype=t)
        s["q_in"], s["k_in"], s["v_in"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["q_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
        s["k_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
        angle = torch.arange(max_seq, device="cuda", dtype=torch.float64)[:, None] * (
            500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
        s["table"] = torch.stack([angle.cos(), angle.sin()], 1).to(torch.float32).contiguous()
        s["n_new"] = _ints(g, (T + 1) // 2, T, B) if case["ragged"] else torch.full((B,), T, dtype=torch.int32, device="cuda")
        s["seq_lens"] = s["n_new"] + (torch.rand(B, generator=g, device="cuda") * (max_seq - s["n_new"] + 1)).to(torch.int32)
        s["seq_lens"] = torch.minimum(s["seq_lens"], torch.full_like(s["seq_lens"], max_seq))
        s["positions"] = None
        if case["positions"]:  # the depth of each drafted token after the context
            depth = _ancestors(_parents(g, B, T))[1] if T <= 128 else torch.arange(T, device="cuda")[None].repeat(B, 1)
            s["positions"] = (depth + (s["seq_lens"] - s["n_new"])[:, None]).to(torch.int32).contiguous()
        s["q_out"] = torch.zeros((B, Hq, T, D), device="cuda", dtype=t)
        s["K"], s["V"], s["bt"] = _cache(case, g, B, Hkv, max_seq, case["bs"])
    elif op == "window_decode":
        B, Hq, Hkv, max_seq = (case[k] for k in ("B", "Hq", "Hkv", "max_seq"))
        s["K"], s["V"], s["bt"] = _cache(case, g, B, Hkv, max_seq, case["bs"])
        s["q"] = torch.randn((B, Hq, D), generator=g, device="cuda", dtype=t)
        s["seq_lens"] = _ints(g, max(1, max_seq // 2), max_seq, B)
        s["out"] = torch.zeros((B, Hq, D), device="cuda", dtype=t)
    elif op == "window_prefill":
        B, Hq, Hkv, L = (case[k] for k in ("B", "Hq", "Hkv", "L"))
        s["q"] = torch.randn((B, Hq, L, D), generator=g, device="cuda", dtype=t)
        s["K"], s["V"], _ = _cache(case, g, B, Hkv, L, 0)
        s["seq_lens"] = _ints(g, (L + 1) // 2, L, B) if case["ragged"] else torch.full((B,), L, dtype=torch.int32, device="cuda")
        s["out"] = torch.zeros((B, Hq, L, D), device="cuda", dtype=t)
    elif op == "tree":
        B, T, Hq, Hkv, L = (case[k] for k in ("B", "T", "Hq", "Hkv", "L"))
        s["K"], s["V"], s["bt"] = _cache(case, g, B, Hkv, L, case["bs"])
        s["q"] = torch.randn((B, Hq, T, D), generator=g, device="cuda", dtype=t)
        s["n_new"] = _ints(g, (T + 1) // 2, T, B) if case["ragged"] else torch.full((B,), T, dtype=torch.int32, device="cuda")
        s["seq_lens"] = torch.maximum(_ints(g, (3 * L + 3) // 4, L, B), s["n_new"])
        s["sees"] = _ancestors(_parents(g, B, T))[0]
        s["mask"] = _bits(s["sees"])
        s["out"] = torch.zeros((B, Hq, T, D), device="cuda", dtype=t)
    elif op == "pages":
        P, F, Hkv, max_seq, bs, r = (case[k] for k in ("parents", "forks", "Hkv", "max_seq", "bs", "r"))
        B, blocks = P * (1 + F), -(-max_seq // bs)
        base = _ints(g, max_seq // 4, max_seq - case["grow"], P)
        n = P * blocks + B * (2 + case["grow"] // bs) + case["spare"]
        perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)[: P * blocks].reshape(P, blocks)
        have = torch.arange(blocks, device="cuda")[None] < ((base + bs - 1) // bs)[:, None]
        s["table"] = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
        s["table"][:P] = torch.where(have, perm, torch.full_like(perm, -1))
        s["ref"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["ref"][perm[have].long()] = 1
        s["seq_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["seq_lens"][:P] = base
        s["base"] = s["seq_lens"].clone()
        row = torch.arange(B, device="cuda", dtype=torch.int32)
        s["parent"] = torch.where(row < P, row, (row - P) % P).to(torch.int32)
        s["new"] = (base[s["parent"].long()] + _ints(g, 1, case["grow"], B)).clamp(max=max_seq).to(torch.int32)
        s["K"] = torch.randn((n, Hkv, bs, D), generator=g, device="cuda", dtype=t)
        s["V"] = torch.randn((n, Hkv, bs, D), generator=g, device="cuda", dtype=t)
        s["codes"] = torch.randint(-2**31, 2**31 - 1, (n, Hkv, bs, r // 32), generator=g, device="cuda", dtype=torch.int32)
    else:
        B, T, Hkv, max_seq, bs, r = (case[k] for k in ("B", "T", "Hkv", "max_seq", "bs", "r"))
        s["K"], s["V"], s["bt"] = _cache(case, g, B, Hkv, max_seq, bs)
        s["codes"] = torch.randint(-2**31, 2**31 - 1, s["K"].shape[:3] + (r // 32,), generator=g, device="cuda", dtype=torch.int32)
        s["n_new"] = torch.full((B,), T, dtype=torch.int32, device="cuda")
        s["seq_lens"] = _ints(g, T, max_seq, B)
        # the first child of the root, then nodes of the later levels (in breadth-first order those come later)
        s["n_keep"] = torch.minimum(_ints(g, 1, case["most"], B), torch.full((B,), T, device="cuda", dtype=torch.int32))
        far = torch.rand((B, T - case["most"]), generator=g, device="cuda").argsort(1)[:, : case["most"] - 1].sort(1)[0] + case["most"]
        keep = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        keep[:, 1:1 + far.shape[1]] = far.to(torch.int32)
        s["n_keep"] = s["n_keep"].clamp(max=1 + far.shape[1])
        s["keep"] = keep
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- the framework's calls


def _dims(s, B, Hq, max_seq):
    import hash_aware_top_b200 as H

    c = s["case"]
    if "dims" not in s:
        s["dims"] = H.dims_for(B, Hq, c["Hkv"], D, c.get("r", 128), max_seq, c["dtype"])
    return H, s["dims"]


def _run_own(s):
    c = s["case"]
    op, bs = c["op"], c.get("bs", 0)
    if op == "norm_rope":
        H, d = _dims(s, c["B"], c["Hq"], c["max_seq"])
        head = (d, s["q_in"], s["k_in"], s["v_in"], s["q_weight"], s["k_weight"], 1e-6, s["table"], c["inter"], s["n_new"],
                s["positions"], s["seq_lens"], s["q_out"], s["K"], s["V"])
        if bs:
            H.hata_norm_rope_paged(*head, s["bt"], bs, s["ws"])
        else:
            H.hata_norm_rope(*head, s["ws"])
        return s["q_out"], s["K"], s["V"]
    if op == "window_decode":
        H, d = _dims(s, c["B"], c["Hq"], c["max_seq"])
        if bs:
            H.hata_window_decode_paged(d, s["q"], s["K"], s["V"], s["bt"], bs, s["seq_lens"], c["window"], c["sink"], 0.0,
                                       s["out"], s["ws"])
        else:
            H.hata_window_decode(d, s["q"], s["K"], s["V"], s["seq_lens"], c["window"], c["sink"], 0.0, s["out"], s["ws"])
        return s["out"]
    if op == "window_prefill":
        H, d = _dims(s, c["B"], c["Hq"], c["L"])
        H.hata_window_prefill(d, s["q"], s["K"], s["V"], s["seq_lens"], c["window"], c["sink"], 0.0, s["out"], s["ws"])
        return s["out"]
    if op == "tree":
        H, d = _dims(s, c["B"], c["Hq"], c["L"])
        if bs:
            H.hata_tree_attention_paged(d, s["q"], s["K"], s["V"], s["bt"], bs, s["seq_lens"], s["n_new"], s["mask"], 0.0,
                                        s["out"], s["ws"])
        else:
            H.hata_tree_attention(d, s["q"], s["K"], s["V"], s["seq_lens"], s["n_new"], s["mask"], 0.0, s["out"], s["ws"])
        return s["out"]
    if op == "pages":
        H, d = _dims(s, s["table"].shape[0], c["Hkv"], c["max_seq"])
        pools = (s["K"], s["V"], s["codes"], s["table"], bs, s["seq_lens"], s["ref"], s["ws"])
        H.hata_pages_resize(d, s["base"], *pools)
        H.hata_pages_fork(d, s["parent"], s["table"], bs, s["seq_lens"], s["ref"], s["ws"])
        H.hata_pages_resize(d, s["new"], *pools)
        return s["K"], s["V"], s["codes"], s["table"], s["seq_lens"], s["ref"]
    H, d = _dims(s, c["B"], c["Hkv"], c["max_seq"])
    H.hata_compact_kv_paged(d, s["keep"], s["n_keep"], s["n_new"], s["seq_lens"], s["K"], s["V"], s["codes"], s["bt"], bs,
                            s["new_lens"], s["ws"])
    return s["K"], s["V"], s["codes"], s["new_lens"]


# ---------------------------------------------------------------- the plain form


def _norm(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight


def _rotate(x, cos, sin, inter):
    """x [B][T][H][D] with cos and sin [B][T][1][rot / 2]."""
    half = cos.shape[-1]
    rot, rest = x[..., : 2 * half], x[..., 2 * half:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if inter else (rot[..., :half], rot[..., half:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1)
    return torch.cat([turned, rest], -1)


def _rows(s, pool, b, pos):
    """Rows `pos` of sequences `b` (index tensors of one shape) of a cache: [..., Hkv, D]."""
    if s["bt"] is None:
        return pool[b, :, pos]
    bs = s["case"]["bs"]
    return pool[s["bt"][b, pos // bs].long(), :, pos % bs]


def _softmax(x):
    """Over the last axis, where -inf is masked; a row with nothing left gives zeros."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _run_plain(s):
    c = s["case"]
    op, t = c["op"], _type(c)
    if op == "norm_rope":
        B, T = c["B"], c["T"]
        start = (s["seq_lens"] - s["n_new"]).long()[:, None]
        i = torch.arange(T, device="cuda")[None]
        valid, slot = i < s["n_new"][:, None], start + i
        pos = slot if s["positions"] is None else s["positions"].long()
        cs = s["table"][pos.clamp(0, s["table"].shape[0] - 1)]
        cos, sin = cs[:, :, 0, None], cs[:, :, 1, None]
        q = _rotate(_norm(s["q_in"], s["q_weight"]), cos, sin, c["inter"]).to(t)
        k = _rotate(_norm(s["k_in"], s["k_weight"]), cos, sin, c["inter"]).to(t)
        s["q_out"].copy_(torch.where(valid[:, None, :, None], q.transpose(1, 2), s["q_out"]))
        b = torch.arange(B, device="cuda")[:, None].expand(B, T)[valid]
        p = slot[valid]
        if s["bt"] is None:
            s["K"][b, :, p], s["V"][b, :, p] = k[valid], s["v_in"][valid]
        else:
            page, off = s["bt"][b, p // c["bs"]].long(), p % c["bs"]
            s["K"][page, :, off], s["V"][page, :, off] = k[valid], s["v_in"][valid]
        return s["q_out"], s["K"], s["V"]
    scale = 1.0 / math.sqrt(D)
    if op == "window_decode":
        B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
        L = s["seq_lens"].long()[:, None]
        n_sink, n_win = min(c["sink"], c["max_seq"]), min(c["window"], c["max_seq"])
        first = torch.arange(n_sink, device="cuda")[None].expand(B, n_sink)
        last = L - n_win + torch.arange(n_win, device="cuda")[None]
        pos = torch.cat([first, last], 1)
        ok = torch.cat([first < L, (last >= n_sink)], 1)
        pos = pos.clamp(0, c["max_seq"] - 1)
        b = torch.arange(B, device="cuda")[:, None].expand_as(pos)
        K, V = _rows(s, s["K"], b, pos).float(), _rows(s, s["V"], b, pos).float()  # [B][n][Hkv][D]
        q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
        x = torch.einsum("bgrd,bngd->bgrn", q, K) * scale
        p = _softmax(x.masked_fill(~ok[:, None, None], -math.inf))
        s["out"].copy_(torch.einsum("bgrn,bngd->bgrd", p, V).reshape(B, Hq, D))
        return s["out"]
    if op == "window_prefill":
        B, Hq, Hkv, L = c["B"], c["Hq"], c["Hkv"], c["L"]
        at = torch.arange(L, device="cuda")
        sees = (at[None] <= at[:, None]) & ((at[None] < c["sink"]) | (at[None] > at[:, None] - c["window"]))
        q = s["q"].float().view(B, Hkv, Hq // Hkv, L, D)
        x = torch.matmul(q, s["K"].float()[:, :, None].transpose(-1, -2)).mul_(scale)
        p = _softmax(x.masked_fill_(~sees, -math.inf))
        o = torch.matmul(p, s["V"].float()[:, :, None]).view(B, Hq, L, D).to(t)
        live = at[None] < s["seq_lens"][:, None]
        s["out"].copy_(torch.where(live[:, None, :, None], o, s["out"]))
        return s["out"]
    if op == "tree":
        B, T, Hq, Hkv, L = c["B"], c["T"], c["Hq"], c["Hkv"], c["L"]
        ctx = (s["seq_lens"] - s["n_new"]).long()[:, None, None]
        at = torch.arange(L, device="cuda")
        if s["bt"] is None:
            K, V = s["K"].float(), s["V"].float()
        else:
            b = torch.arange(B, device="cuda")[:, None].expand(B, L)
            K, V = (_rows(s, s[k], b, at[None].expand(B, L)).float().transpose(1, 2) for k in ("K", "V"))
        node = at[None, None] - ctx  # which drafted token a slot holds
        known = torch.gather(s["sees"], 2, node.clamp(0, T - 1).expand(B, T, L))
        sees = (node < 0) | (known & (node < s["n_new"][:, None, None]))
        q = s["q"].float().view(B, Hkv, (Hq // Hkv) * T, D)
        x = torch.matmul(q, K.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, T, L) * scale
        p = _softmax(x.masked_fill(~sees[:, None, None], -math.inf))
        o = torch.matmul(p.view(B, Hkv, -1, L), V).view(B, Hq, T, D).to(t)
        live = torch.arange(T, device="cuda")[None] < s["n_new"][:, None]
        s["out"].copy_(torch.where(live[:, None, :, None], o, s["out"]))
        return s["out"]
    if op == "pages":
        _resize_plain(s, s["base"])
        blocks, B = s["table"].shape[1], s["table"].shape[0]
        rows = torch.arange(B, device="cuda")
        changed = s["parent"].long() != rows
        new = s["table"][s["parent"].long()]
        n = s["ref"].shape[0]
        gone = torch.bincount(torch.where(changed[:, None] & (s["table"] >= 0), s["table"], n).flatten(), minlength=n + 1)[:n]
        came = torch.bincount(torch.where(changed[:, None] & (new >= 0), new, n).flatten(), minlength=n + 1)[:n]
        s["ref"].add_((came - gone).to(torch.int32))
        s["table"].copy_(new)
        s["seq_lens"].copy_(s["seq_lens"][s["parent"].long()])
        _resize_plain(s, s["new"])
        return s["K"], s["V"], s["codes"], s["table"], s["seq_lens"], s["ref"]
    B, T, bs = c["B"], c["T"], c["bs"]
    j = torch.arange(T, device="cuda")[None]
    ok = j < s["n_keep"][:, None]
    base = (s["seq_lens"] - s["n_new"]).long()[:, None]
    b = torch.arange(B, device="cuda")[:, None].expand(B, T)[ok]
    src, dst = (base + s["keep"].long())[ok], (base + j)[ok]
    for name in ("K", "V", "codes"):
        pool = s[name]
        pool[s["bt"][b, dst // bs].long(), :, dst % bs] = pool[s["bt"][b, src // bs].long(), :, src % bs]
    s["new_lens"].copy_(s["seq_lens"] - s["n_new"] + s["n_keep"])
    return s["K"], s["V"], s["codes"], s["new_lens"]


def _resize_plain(s, new):
    """Pages freed, copied on write where a shared page would be written, and allocated, lowest free page first."""
    bs, table, ref = s["case"]["bs"], s["table"], s["ref"]
    (B, blocks), n = table.shape, ref.shape[0]
    old, new = s["seq_lens"].long(), new.long()
    col = torch.arange(blocks, device="cuda")[None]
    n_old, n_new = (old + bs - 1) // bs, (new + bs - 1) // bs
    drop = (col >= n_new[:, None]) & (col < n_old[:, None])
    ref.sub_(torch.bincount(torch.where(drop, table, n).flatten(), minlength=n + 1)[:n].to(torch.int32))
    table.masked_fill_(drop, -1)
    # a growing sequence whose last page is partly filled and shared gets a page of its own; the last sharer keeps it
    grows = (new > old) & (old % bs != 0)
    tail = torch.gather(table, 1, (n_old - 1).clamp(min=0)[:, None])[:, 0].long()
    page = torch.where(grows, tail, -1 - torch.arange(B, device="cuda"))
    before = ((page[None] == page[:, None]) & (torch.arange(B, device="cuda")[None] < torch.arange(B, device="cuda")[:, None])).sum(1)
    copy = grows & (ref[tail.clamp(min=0)] - before > 1)
    first = torch.where(copy, n_old - 1, n_old)
    want = (col >= first[:, None]) & (col < n_new[:, None])
    order = torch.argsort((ref != 0).to(torch.int8), stable=True).to(torch.int32)  # free pages first, the lowest first
    rank = (want.flatten().cumsum(0) - 1).clamp(min=0).view(B, blocks)
    table.copy_(torch.where(want, order[rank.clamp(max=n - 1)], table))
    ref.sub_(torch.bincount(torch.where(copy, tail, n), minlength=n + 1)[:n].to(torch.int32))
    ref.add_(torch.bincount(torch.where(want, table, n).flatten(), minlength=n + 1)[:n].to(torch.int32))
    to = torch.gather(table, 1, (n_old - 1).clamp(min=0)[:, None])[:, 0].long()
    rows = (torch.arange(bs, device="cuda")[None] < (old % bs)[:, None])[copy][:, None, :, None]
    for name in ("K", "V", "codes"):
        s[name][to[copy]] = torch.where(rows, s[name][tail[copy]], s[name][to[copy]])
    s["seq_lens"].copy_(new)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work


def _mean_len(lo, hi):
    return (lo + hi) / 2


def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "norm_rope":
        n = case["B"] * (_mean_len((case["T"] + 1) // 2, case["T"]) if case["ragged"] else case["T"])
        rows = n * (case["Hq"] + 2 * case["Hkv"])
        return {"bytes": 2 * rows * D * e + n * case["rot"] * 4, "flops": 6 * n * (case["Hq"] + case["Hkv"]) * D}
    if op == "window_decode":
        L = _mean_len(max(1, case["max_seq"] // 2), case["max_seq"])
        n = min(L, case["window"] + case["sink"])
        B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
        return {"bytes": 2 * B * Hkv * n * D * e + 2 * B * Hq * D * e, "flops": 4 * B * Hq * n * D}
    if op == "window_prefill":
        B, Hq, Hkv, top, w, k = (case[x] for x in ("B", "Hq", "Hkv", "L", "window", "sink"))
        L = _mean_len((top + 1) // 2, top) if case["ragged"] else top
        near = L * (L + 1) / 2 - max(0, L - w) * (max(0, L - w) + 1) / 2  # pairs inside the window
        m = max(0, L - w)  # rows whose window no longer reaches the first token: t = w .. L - 1 see min(k, t - w + 1) more
        far = m * (m + 1) / 2 - max(0, m - k) * (max(0, m - k) + 1) / 2
        return {"bytes": (2 * Hq + 2 * Hkv) * B * L * D * e, "flops": 4 * B * Hq * (near + far) * D}
    if op == "tree":
        B, T, Hq, Hkv, top = (case[x] for x in ("B", "T", "Hq", "Hkv", "L"))
        L, T = _mean_len((3 * top + 3) // 4, top), _mean_len((T + 1) // 2, T) if case["ragged"] else T
        return {"bytes": 2 * B * Hkv * L * D * e + 2 * B * Hq * T * D * e, "flops": 4 * B * Hq * T * L * D}
    row = case["Hkv"] * (2 * D * e + case["r"] // 8)
    if op == "pages":
        B, blocks = case["parents"] * (1 + case["forks"]), -(-case["max_seq"] // case["bs"])
        pages = case["parents"] * blocks + B * (2 + case["grow"] // case["bs"]) + case["spare"]
        copies = case["parents"] * case["forks"] * case["bs"] / 2  # rows of half a page for each fork
        return {"bytes": 2 * copies * row + 2 * 4 * (B * blocks + pages), "flops": 0}
    return {"bytes": 2 * case["B"] * (case["most"] + 1) / 2 * row, "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits


def _seen_rows(s, name, b, at):
    """Rows `at` (a 1-D index) of sequence b in 64 bits: [Hkv][n][D]."""
    if s.get("bt") is None:
        return s[name][b, :, at].double()
    bs = s["case"]["bs"]
    return s[name][s["bt"][b].long()[at // bs], :, at % bs].double().transpose(0, 1)


def _attend(q, K, V, sees):
    """q [H][n][D] against K, V [Hkv][m][D] with sees [n][m] (or None)."""
    out = torch.zeros_like(q)
    G = q.shape[0] // K.shape[0]
    for h in range(q.shape[0]):
        x = q[h] @ K[h // G].T / math.sqrt(D)
        if sees is not None:
            x = x.masked_fill(~sees, -math.inf)
            dead = ~sees.any(-1, keepdim=True)
            out[h] = torch.softmax(x.masked_fill(dead, 0.0), -1).masked_fill(dead, 0.0) @ V[h // G]
        else:
            out[h] = torch.softmax(x, -1) @ V[h // G]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        q_out, K, V = s["q_out"].double(), s["K"].double(), s["V"].double()
        half = case["rot"] // 2
        first = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
        second = first + (1 if case["inter"] else half)
        for b in range(case["B"]):
            n, L = int(s["n_new"][b]), int(s["seq_lens"][b])
            slot = torch.arange(L - n, L, device="cuda")
            pos = slot if s["positions"] is None else s["positions"][b, :n].long()
            z = torch.complex(s["table"][pos, 0].double(), s["table"][pos, 1].double())[:, None]
            for x, w, what in ((s["q_in"], s["q_weight"], "q"), (s["k_in"], s["k_weight"], "k"), (s["v_in"], None, "v")):
                y = x[b, :n].double()
                if w is not None:
                    y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
                    u = torch.complex(y[..., first], y[..., second]) * z
                    y[..., first], y[..., second] = u.real, u.imag
                if what == "q":
                    q_out[b, :, :n] = y.transpose(0, 1)
                else:
                    to = K if what == "k" else V
                    if s["bt"] is None:
                        to[b, :, L - n:L] = y.transpose(0, 1)
                    else:
                        to[s["bt"][b].long()[slot // case["bs"]], :, slot % case["bs"]] = y
        return q_out, K, V
    if op == "window_decode":
        out = s["out"].double()
        for b in range(case["B"]):
            L = int(s["seq_lens"][b])
            at = torch.arange(L, device="cuda")
            at = at[(at < case["sink"]) | (at >= L - case["window"])]
            out[b] = _attend(s["q"][b, :, None].double(), _seen_rows(s, "K", b, at), _seen_rows(s, "V", b, at), None)[:, 0]
        return out
    if op == "window_prefill":
        out = s["out"].double()
        for b in range(case["B"]):
            L = int(s["seq_lens"][b])
            far = torch.arange(L, device="cuda")[:, None] - torch.arange(L, device="cuda")[None]
            sees = (far >= 0) & ((far < case["window"]) | (torch.arange(L, device="cuda")[None] < case["sink"]))
            out[b, :, :L] = _attend(s["q"][b, :, :L].double(), s["K"][b, :, :L].double(), s["V"][b, :, :L].double(), sees)
        return out
    if op == "tree":
        out = s["out"].double()
        for b in range(case["B"]):
            n, L = int(s["n_new"][b]), int(s["seq_lens"][b])
            at = torch.arange(L, device="cuda")
            sees = torch.ones((n, L), dtype=torch.bool, device="cuda")
            sees[:, L - n:] = s["sees"][b, :n, :n]
            out[b, :, :n] = _attend(s["q"][b, :, :n].double(), _seen_rows(s, "K", b, at), _seen_rows(s, "V", b, at), sees)
        return out
    if op == "pages":
        return _exact_pages(s)
    for b in range(case["B"]):
        n, L = int(s["n_new"][b]), int(s["seq_lens"][b])
        bs, pages = case["bs"], s["bt"][b].tolist()
        for name in ("K", "V", "codes"):
            rows = [s[name][pages[p // bs], :, p % bs].clone() for p in (L - n + k for k in s["keep"][b, : int(s["n_keep"][b])].tolist())]
            for j, row in enumerate(rows):
                s[name][pages[(L - n + j) // bs], :, (L - n + j) % bs] = row
        s["new_lens"][b] = L - n + int(s["n_keep"][b])
    return s["K"].double(), s["V"].double(), None, None


def _exact_pages(s):
    """The beam step on lists, sequence by sequence."""
    bs, ref, blocks = s["case"]["bs"], s["ref"].tolist(), s["table"].shape[1]
    pages = [[p for p in row if p >= 0] for row in s["table"].tolist()]
    lens, new = s["base"].tolist(), s["new"].tolist()
    pages_before = [list(p) for p in pages]
    for b, parent in enumerate(s["parent"].tolist()):
        if parent != b:
            for p in pages_before[b]:
                ref[p] -= 1
            for p in pages_before[parent]:
                ref[p] += 1
            pages[b], lens[b] = list(pages_before[parent]), s["base"].tolist()[parent]
    free = [p for p in range(len(ref)) if ref[p] == 0]
    for b in range(len(pages)):
        if new[b] > lens[b] and lens[b] % bs and ref[pages[b][-1]] > 1:
            src, dst = pages[b][-1], free.pop(0)
            for name in ("K", "V", "codes"):
                s[name][dst, :, : lens[b] % bs] = s[name][src, :, : lens[b] % bs]
            ref[src] -= 1
            ref[dst] += 1
            pages[b][-1] = dst
        while len(pages[b]) * bs < new[b]:
            pages[b].append(free.pop(0))
            ref[pages[b][-1]] += 1
    return s["K"].double(), s["V"].double(), None, None, None, None
