"""Page bookkeeping (hata_pages_fork, hata_pages_resize) and row compaction (hata_compact_kv, _paged) against a
model on Python lists, and a whole serving round over a paged cache."""
import ctypes

import numpy as np
import pytest
import torch

D = 128


@pytest.fixture(scope="module")
def H():
    import hash_aware_top_b200 as H

    return H


class Model:
    """A paged cache on lists: pages hold one number per slot, which stands for the slot's K, V and code rows."""

    def __init__(self, B, n_blocks, bs, max_seq):
        self.bs, self.max_seq = bs, max_seq
        self.pages, self.lens, self.ref = [[] for _ in range(B)], [0] * B, [0] * n_blocks

    def fork(self, parent):
        old_pages, old_lens = [list(p) for p in self.pages], list(self.lens)
        for b, pa in enumerate(parent):
            if 0 <= pa < len(parent) and pa != b:
                for p in old_pages[b]:
                    self.ref[p] -= 1
                for p in old_pages[pa]:
                    self.ref[p] += 1
                self.pages[b], self.lens[b] = list(old_pages[pa]), old_lens[pa]

    def resize(self, new):
        """Copies (source, target, rows) that were made; None if the pool had too few pages for the growth."""
        bs = self.bs
        new = [n if 0 <= n <= self.max_seq else self.lens[b] for b, n in enumerate(new)]
        for b, n in enumerate(new):
            while len(self.pages[b]) > -(-n // bs):
                self.ref[self.pages[b].pop()] -= 1
            if n < self.lens[b]:
                self.lens[b] = n
        pages, ref, copies = [list(p) for p in self.pages], list(self.ref), []
        free = [p for p, r in enumerate(ref) if r == 0]
        for b, n in enumerate(new):
            if n <= self.lens[b]:
                continue
            if self.lens[b] % bs and ref[pages[b][-1]] > 1:
                if not free:
                    return None
                src, dst = pages[b][-1], free.pop(0)
                copies.append((src, dst, self.lens[b] % bs))
                ref[src] -= 1
                ref[dst] += 1
                pages[b][-1] = dst
            while len(pages[b]) * bs < n:
                if not free:
                    return None
                pages[b].append(free.pop(0))
                ref[pages[b][-1]] += 1
        self.pages, self.ref, self.lens = pages, ref, list(new)
        return copies


class Cache:
    def __init__(self, H, B, n_blocks, bs, max_seq, Hkv=2, r=128, dtype=torch.bfloat16, codes=True, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.bs = H, bs
        self.d = H.dims_for(B, Hkv, Hkv, D, r, max_seq, dtype)
        self.K = torch.randn(n_blocks, Hkv, bs, D, generator=g, device="cuda").to(dtype)
        self.V = torch.randn(n_blocks, Hkv, bs, D, generator=g, device="cuda").to(dtype)
        shape, wide = self.d.code_shape(n_blocks, Hkv, bs), r != 16
        self.codes = torch.randint(-2**15, 2**15, shape, generator=g, device="cuda",
                                   dtype=torch.int32 if wide else torch.int16) if codes else None
        self.table = torch.full((B, -(-max_seq // bs)), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(H.hata_pages_workspace_size(self.d), dtype=torch.uint8, device="cuda")

    def fork(self, parent):
        self.H.hata_pages_fork(self.d, torch.tensor(parent, dtype=torch.int32, device="cuda"), self.table, self.bs, self.lens,
                               self.ref, self.ws)

    def resize(self, new):
        self.H.hata_pages_resize(self.d, torch.tensor(new, dtype=torch.int32, device="cuda"), self.K, self.V, self.codes,
                                 self.table, self.bs, self.lens, self.ref, self.ws)

    def status(self):
        return self.H.hata_read_device_status(self.ws)

    def tensors(self):
        return [t for t in (self.K, self.V, self.codes) if t is not None]

    def same_as(self, m):
        assert self.lens.tolist() == m.lens
        assert self.ref.tolist() == m.ref
        want = [p + [-1] * (self.table.shape[1] - len(p)) for p in m.pages]
        assert self.table.tolist() == want


@pytest.mark.gpu
@pytest.mark.parametrize("B,n_blocks,bs,max_seq,r,dtype", [
    (1, 3, 16, 48, 128, torch.bfloat16), (7, 60, 16, 200, 32, torch.float32), (33, 300, 16, 334, 16, torch.bfloat16),
    (4, 40, 64, 500, 256, torch.bfloat16), (3, 9, 1024, 2500, 64, torch.float32), (1024, 5000, 16, 64, 128, torch.bfloat16),
])
def test_random_steps_follow_the_model(H, B, n_blocks, bs, max_seq, r, dtype):
    """Forks, growth with copies on write, shrinking and refused growth in random order."""
    rng = np.random.default_rng(B + bs)
    c, m = Cache(H, B, n_blocks, bs, max_seq, r=r, dtype=dtype, Hkv=1 if B > 500 else 2), Model(B, n_blocks, bs, max_seq)
    refused = 0
    for step in range(12):
        if step % 3 == 2:
            parent = rng.integers(-1, B, B).tolist()
            c.fork(parent)
            m.fork(parent)
        else:
            new = [int(x) for x in rng.integers(0, max_seq + 1, B)]
            if step % 2:  # mostly small changes
                new = [max(0, min(max_seq, old + int(rng.integers(-5, 20)))) for old in m.lens]
            before = [t.clone() for t in c.tensors()]
            c.resize(new)
            copies = m.resize(new)
            refused += copies is None
            assert c.status() == (H.HATA_ERR_NO_PAGES if copies is None else 0)
            for src, dst, rows in copies or []:
                for t in before:
                    t[dst, :, :rows] = t[src, :, :rows]
            for got, want in zip(c.tensors(), before):
                assert torch.equal(got, want)
        c.same_as(m)
    c.resize([0] * B)
    m.resize([0] * B)
    c.same_as(m)
    assert sum(m.ref) == 0


@pytest.mark.gpu
def test_a_pool_whose_counts_do_not_fit_shared_memory(H):
    """70,000 pages: the counts stay in global memory."""
    rng = np.random.default_rng(5)
    B, n_blocks = 6, 70000
    c = Cache(H, B, 8, 16, 4000, Hkv=1, codes=False)
    c.K = torch.zeros(n_blocks, 1, 16, D, device="cuda", dtype=torch.bfloat16)
    c.V, c.ref = c.K.clone(), torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
    m = Model(B, n_blocks, 16, 4000)
    for step in range(6):
        if step % 3 == 1:
            parent = rng.integers(-1, B, B).tolist()
            c.fork(parent), m.fork(parent)
        else:
            new = [int(x) for x in rng.integers(0, 4001, B)]
            c.resize(new)
            assert m.resize(new) is not None
        assert c.status() == 0
        c.same_as(m)


@pytest.mark.gpu
def test_growing_sharers_copy_and_the_last_keeps(H):
    c, m = Cache(H, 4, 12, 16, 100), Model(4, 12, 16, 100)
    for step in ([20, 0, 0, 0], "fork", [21, 25, 21, 40]):
        if step == "fork":
            c.fork([0, 0, 0, 0])
            m.fork([0, 0, 0, 0])
        else:
            c.resize(step)
            m.resize(step)
        c.same_as(m)
    assert m.pages[3][1] == 1 and len({p[1] for p in m.pages}) == 4 and {p[0] for p in m.pages} == {0}


@pytest.mark.gpu
def test_too_few_pages_leave_lengths(H):
    c, m = Cache(H, 3, 4, 16, 64), Model(3, 4, 16, 64)
    c.resize([16, 40, 0]), m.resize([16, 40, 0])
    c.resize([17, 10, 64]), m.resize([17, 10, 64])  # shrinking still happens
    assert c.status() == H.HATA_ERR_NO_PAGES
    c.same_as(m)
    assert m.lens == [16, 10, 0]


@pytest.mark.gpu
def test_bad_lengths_and_parents_are_flagged(H):
    c, m = Cache(H, 3, 10, 16, 64), Model(3, 10, 16, 64)
    c.resize([20, 65, -1]), m.resize([20, 65, -1])
    assert c.status() == H.HATA_ERR_INVALID_ARG
    c.same_as(m)
    c.fork([0, 3, -5]), m.fork([0, 3, -5])
    assert c.status() == H.HATA_ERR_INVALID_ARG
    c.same_as(m)
    # a table entry outside the pool and a count that is too low: flagged, nothing outside is touched
    c.table[0, 1] = 99
    c.ref[c.table[0, 0].long()] = 0
    c.resize([0, 0, 0])
    assert c.status() == H.HATA_ERR_INVALID_ARG
    assert c.ref.min() >= 0 and c.lens.tolist() == [0, 0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("T,r,dtype,codes", [(1, 128, torch.bfloat16, True), (64, 32, torch.float32, True),
                                             (128, 16, torch.bfloat16, True), (700, 256, torch.bfloat16, True),
                                             (9, 64, torch.float32, False)])
def test_compact(H, paged, T, r, dtype, codes):
    B, Hkv, max_seq, bs = 5, 2, 720, 16
    rng = np.random.default_rng(T)
    d = H.dims_for(B, Hkv, Hkv, D, r, max_seq, dtype)
    nb = max_seq // bs
    lead = (B * nb, Hkv, bs) if paged else (B, Hkv, max_seq)
    bt = torch.randperm(B * nb, device="cuda").int().view(B, nb).contiguous()
    tensors = [torch.randn(*lead, D, device="cuda").to(dtype), torch.randn(*lead, D, device="cuda").to(dtype)]
    if codes:
        tensors.append(torch.randint(-2**15, 2**15, d.code_shape(*lead), device="cuda",
                                     dtype=torch.int32 if r != 16 else torch.int16))
    n_new = np.array([T, max(T // 2, 1), T, T, 0], dtype=np.int32)
    n_keep = np.array([n_new[0], n_new[1] // 2, 0, rng.integers(1, T + 1), 0], dtype=np.int32)
    lens = np.array([rng.integers(n, max_seq + 1) for n in n_new], dtype=np.int32)
    keep = np.full((B, T), -7, dtype=np.int32)
    for b in range(B):
        keep[b, :n_keep[b]] = np.sort(rng.choice(max(n_new[b], 1), n_keep[b], replace=False))
    want = [t.clone() for t in tensors]
    for b in range(B):
        base = lens[b] - n_new[b]
        for j in range(n_keep[b]):
            s, t2 = base + keep[b, j], base + j
            for t, w in zip(tensors, want):
                if paged:
                    w[bt[b, t2 // bs].long(), :, t2 % bs] = t[bt[b, s // bs].long(), :, s % bs]
                else:
                    w[b, :, t2] = t[b, :, s]
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    args = (d, dev(keep), dev(n_keep), dev(n_new), dev(lens), tensors[0], tensors[1], tensors[2] if codes else None)
    if paged:
        H.hata_compact_kv_paged(*args, bt, bs, new_lens, ws)
    else:
        H.hata_compact_kv(*args, new_lens, ws)
    assert H.hata_read_device_status(ws) == 0
    for got, w in zip(tensors, want):
        assert torch.equal(got, w)
    assert new_lens.tolist() == (lens - n_new + n_keep).tolist()


@pytest.mark.gpu
def test_compact_leaves_bad_sequences(H):
    B, T, max_seq = 6, 4, 32
    d = H.dims_for(B, 1, 1, D, 32, max_seq, "f32")
    K = torch.randn(B, 1, max_seq, D, device="cuda")
    V, K0 = K.clone(), K.clone()
    keep = torch.tensor([[1, 1, 2, 3], [3, 2, 0, 0], [0, 4, 0, 0], [-1, 0, 0, 0], [1, 2, 3, 3], [1, 3, 0, 0]],
                        dtype=torch.int32, device="cuda")
    n_keep = torch.tensor([2, 2, 2, 1, 5, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([9, 9, 9, 9, 9, 3], dtype=torch.int32, device="cuda")  # the last is shorter than its 4 tokens
    new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    H.hata_compact_kv(d, keep, n_keep, None, lens, K, V, None, new_lens, ws)
    assert H.hata_read_device_status(ws) == H.HATA_ERR_INVALID_ARG
    assert torch.equal(K, K0) and torch.equal(V, K0) and torch.equal(new_lens, lens)


def test_refusals(H):
    P = ctypes.c_void_p
    f, odd, null = P(0x1000), P(0x1008), P(0)
    d = H.dims_for(2, 4, 2, D, 128, 64, "bf16")
    big = H.dims_for(1025, 4, 2, D, 128, 64, "bf16")
    n = ctypes.c_size_t(0)
    assert H.lib.hata_pages_workspace_size(ctypes.byref(big), ctypes.byref(n)) == 2
    assert H.lib.hata_pages_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    fork = lambda dd=d, pa=f, bt=f, bs=16, nb=4, ref=f, ws=f, wsb=n.value: H.lib.hata_pages_fork(  # noqa: E731
        ctypes.byref(dd), pa, bt, bs, nb, f, ref, ws, wsb, null)
    assert fork(pa=null) == 1 and fork(bt=null) == 1 and fork(bs=17) == 1 and fork(nb=0) == 1 and fork(ref=null) == 1
    assert fork(dd=big, wsb=1 << 20) == 2 and fork(ws=null) == 5 and fork(ws=odd) == 5 and fork(wsb=n.value - 1) == 5
    size = lambda dd=d, new=f, K=f, codes=f, bt=f, bs=16, nb=4, ws=f, wsb=n.value: H.lib.hata_pages_resize(  # noqa: E731
        ctypes.byref(dd), new, K, f, codes, bt, bs, nb, f, f, ws, wsb, null)
    assert size(new=null) == 1 and size(K=odd) == 1 and size(codes=odd) == 1 and size(bt=null) == 1 and size(bs=8) == 1
    assert size(dd=big, wsb=1 << 20) == 2 and size(ws=null) == 5 and size(wsb=16) == 5
    comp = lambda T=4, keep=f, K=f, codes=null, lens=P(0x2000), new=f, ws=f, wsb=16: H.lib.hata_compact_kv(  # noqa: E731
        ctypes.byref(d), T, keep, f, null, lens, K, f, codes, new, ws, wsb, null)
    assert comp(T=0) == 1 and comp(T=65) == 1 and comp(keep=null) == 1 and comp(K=odd) == 1 and comp(codes=odd) == 1
    assert comp(lens=null) == 1 and comp(new=P(0x2000)) == 1 and comp(ws=null) == 5 and comp(wsb=8) == 5
    assert H.lib.hata_compact_kv_paged(ctypes.byref(d), 4, f, f, null, P(0x2000), f, f, null, null, 16, 4, f, f, 16, null) == 1
    assert H.hata_status_string(H.HATA_ERR_NO_PAGES) == "too few free pages in the pool"


def test_compact_refuses_new_lens_over_its_inputs(H):
    """new_lens is written while other CTAs still read keep, n_keep, n_new, seq_lens and the table."""
    P = ctypes.c_void_p
    f, null, d = P(0x100000), P(0), H.dims_for(5, 4, 2, D, 128, 64, "bf16")
    at = dict(keep=0x1000, n_keep=0x2000, n_new=0x3000, lens=0x4000, table=0x5000, new=0x6000)  # 80, 20, 20, 20, 80 bytes

    def call(paged, **kw):
        a = {k: P(v) for k, v in {**at, **kw}.items()}
        head = (ctypes.byref(d), 4, a["keep"], a["n_keep"], a["n_new"], a["lens"], f, f, f)
        if paged:
            return H.lib.hata_compact_kv_paged(*head, a["table"], 16, 4, a["new"], f, 16, null)
        return H.lib.hata_compact_kv(*head, a["new"], f, 16, null)

    for paged in (False, True):
        for name, size in (("keep", 80), ("n_keep", 20), ("n_new", 20), ("lens", 20)):
            for off in (-16, 0, 4, size - 4):
                assert call(paged, new=at[name] + off) == 1, (paged, name, off)
    assert call(True, new=at["table"]) == 1 and call(True, new=at["table"] + 76) == 1


def pad(rows, T):
    return torch.tensor([r + [0] * (T - len(r)) for r in rows], dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,r", [(torch.bfloat16, 128), (torch.float32, 16)])
def test_compact_leaves_rows_that_another_sequence_holds(H, dtype, r):
    """After a fork the drafted rows lie in pages of several sequences: a sequence that would move some of them is flagged
    and left; one that moves nothing, or only rows past the other's end, is not."""
    B, T, bs = 5, 6, 16
    c = Cache(H, B, 40, bs, 100, r=r, dtype=dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def compact(keep, n_new):
        c.H.hata_compact_kv_paged(c.d, pad(keep, T), i32([len(k) for k in keep]), i32(n_new), c.lens, c.K, c.V, c.codes, c.table, bs,
                                  new_lens, ws)
        return c.H.hata_read_device_status(ws)

    def rows(t, b, n):
        at = torch.arange(n, device="cuda")
        return t[c.table[b].long()[at // bs], :, at % bs]

    def held(lens):
        return [[rows(t, b, n).clone() for b, n in enumerate(lens)] for t in c.tensors()]

    c.resize([0, 45, 38, 30, 0])
    c.fork([1, 1, 2, 3, 3])  # 0 and 1 share pages, 3 and 4 do
    assert c.lens.tolist() == [45, 45, 38, 30, 30] and c.status() == 0
    before = held(c.lens.tolist())
    # 0 and 1 keep other paths of shared rows, 2 is alone, 3 moves nothing, 4 keeps nothing
    assert compact([[0, 2, 5], [1, 3], [1, 4, 5], [0, 1, 2], []], [6, 6, 6, 6, 6]) == H.HATA_ERR_INVALID_ARG
    assert new_lens.tolist() == [45, 45, 35, 27, 24]
    for old, t in zip(before, c.tensors()):
        for b in (0, 1, 3, 4):
            assert torch.equal(rows(t, b, len(old[b])), old[b])
        assert torch.equal(rows(t, 2, 35), torch.cat([old[2][:32], old[2][[33, 36, 37]]]))
    # the other holds the page, but not the rows that move: 4 goes back to 25 rows, 3 keeps rows 25 to 29 in other places
    c.resize([45, 45, 35, 30, 25])
    before = held([45, 45, 35, 30, 25])
    assert compact([[], [], [], [1, 3], []], [0, 0, 0, 5, 0]) == 0 and new_lens.tolist() == [45, 45, 35, 27, 25]
    for old, t in zip(before, c.tensors()):
        assert torch.equal(rows(t, 3, 27), torch.cat([old[3][:25], old[3][[26, 28]]]))
        assert torch.equal(rows(t, 4, 25), old[4][:25])
    # a first moved row below the other's end is one too many
    assert compact([[], [], [], [1, 3], []], [0, 0, 0, 6, 0]) == H.HATA_ERR_INVALID_ARG and new_lens.tolist()[3] == 30
    # and entries past a sequence's end hold nothing
    c.resize([45, 0, 35, 30, 0])
    c.table[1] = c.table[0]
    c.table[4] = c.table[3]
    assert compact([[2], [], [], [5], []], [6, 0, 0, 6, 0]) == 0 and new_lens.tolist() == [40, 0, 35, 25, 0]


@pytest.mark.gpu
def test_beams_that_fork_then_grow_keep_their_own_paths(H):
    """Fork first, then grow: every beam's drafted rows are its own, and each keeps another path."""
    B, T, bs, L = 4, 5, 16, 27
    c = Cache(H, B, 30, bs, 64)
    c.resize([L, 0, 0, 0])
    c.fork([0, 0, 0, 0])
    c.resize([L + T] * B)
    at = torch.arange(L + T, device="cuda")
    place = [(c.table[b].long()[at // bs], at % bs) for b in range(B)]
    for t in c.tensors():  # the drafted rows of each beam
        for b in range(B):
            page, off = place[b][0][L:], place[b][1][L:]
            t[page, :, off] = (torch.arange(b * T, (b + 1) * T, device="cuda")[:, None, None]).expand(T, t.shape[1], t.shape[3]).to(t.dtype)
    want = [[t[p, :, o].clone() for p, o in place] for t in c.tensors()]
    keep = [[0, 2], [1, 2, 4], [4], [0, 1, 2, 3, 4]]
    new_lens, ws = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(16, dtype=torch.uint8, device="cuda")
    H.hata_compact_kv_paged(c.d, pad(keep, T), torch.tensor([len(k) for k in keep], dtype=torch.int32, device="cuda"), None, c.lens,
                            c.K, c.V, c.codes, c.table, bs, new_lens, ws)
    assert H.hata_read_device_status(ws) == 0 and new_lens.tolist() == [L + len(k) for k in keep]
    for t, w in zip(c.tensors(), want):
        for b, (p, o) in enumerate(place):
            n = L + len(keep[b])
            assert torch.equal(t[p[:n], :, o[:n]], torch.cat([w[b][:L], w[b][L:][keep[b]]]))


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,Hkv,r,dtype", [(300, 3, 16, torch.bfloat16), (210, 2, 64, torch.float32), (260, 5, 256, torch.bfloat16)])
def test_compact_of_many_sequences(H, paged, B, Hkv, r, dtype):
    """So many that a CTA takes several heads, odd numbers of heads among them."""
    T, max_seq, bs = 40, 64, 16
    g = torch.Generator().manual_seed(B)
    d = H.dims_for(B, Hkv, Hkv, D, r, max_seq, dtype)
    nb = max_seq // bs
    lead = (B * nb, Hkv, bs) if paged else (B, Hkv, max_seq)
    bt = torch.randperm(B * nb, generator=g).int().view(B, nb).cuda()
    tensors = [torch.randn(*lead, D, device="cuda").to(dtype), torch.randn(*lead, D, device="cuda").to(dtype),
               torch.randint(-2**15, 2**15, d.code_shape(*lead), device="cuda", dtype=torch.int32 if r != 16 else torch.int16)]
    lens = torch.randint(T, max_seq + 1, (B,), generator=g)
    n_keep = torch.randint(0, T + 1, (B,), generator=g)
    keep = torch.stack([torch.cat([torch.randperm(T, generator=g)[:n].sort()[0], torch.full((T - n,), -1)]) for n in n_keep.tolist()])
    b = torch.arange(B)[:, None].expand(B, T)
    j = torch.arange(T)[None].expand(B, T)
    ok = j < n_keep[:, None]
    b, src, dst = b[ok].cuda(), ((lens - T)[:, None] + keep)[ok].cuda(), ((lens - T)[:, None] + j)[ok].cuda()
    want = [t.clone() for t in tensors]
    for t, w in zip(tensors, want):
        if paged:
            w[bt[b, dst // bs].long(), :, dst % bs] = t[bt[b, src // bs].long(), :, src % bs]
        else:
            w[b, :, dst] = t[b, :, src]
    new_lens, ws = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(16, dtype=torch.uint8, device="cuda")
    args = (d, keep.int().cuda(), n_keep.int().cuda(), None, lens.int().cuda(), *tensors)
    if paged:
        H.hata_compact_kv_paged(*args, bt, bs, new_lens, ws)
    else:
        H.hata_compact_kv(*args, new_lens, ws)
    assert H.hata_read_device_status(ws) == 0 and new_lens.tolist() == (lens - T + n_keep).tolist()
    for got, w in zip(tensors, want):
        assert torch.equal(got, w)
