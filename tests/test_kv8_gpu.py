"""The operators over the 8-bit key / value cache against plain 64-bit forms (tests/kv8_util.py, which
also derives the bounds), through the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv8_util as ref

pytestmark = pytest.mark.gpu
BLOCK = 32


@pytest.fixture(scope="module")
def uocr(cuda_device):
    import block_sparse_long_uocr_b200 as m
    return m


def to(dev, *tensors):
    """Copies on the device (also when it is the CPU's)."""
    return [t.clone().to(dev) for t in tensors]


class Case:
    """Caches, tables and queries on the CPU; rows behind a sequence's end hold the code of NaN."""

    def __init__(self, lens, H, seed, n_q=None, max_blocks=None, odd_scale=False, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.g = lens, H, g
        self.mb = max_blocks or max(1, max(-(-max(x, 0) // BLOCK) for x in lens))
        self.table, pages = ref.make_table(g, lens, self.mb)
        self.k, self.ks = ref.make_pool(g, pages, H, odd_scale=odd_scale)
        self.v, self.vs = ref.make_pool(g, pages, H, odd_scale=odd_scale)
        for b, x in enumerate(lens):
            if x > 0 and x % BLOCK:
                for c in (self.k, self.v):
                    c.view(torch.uint8)[int(self.table[b, x // BLOCK]), :, x % BLOCK:] = 0x7F
        n = len(lens) if n_q is None else n_q
        self.q = (torch.randn((n, H, 128), generator=g) * q_scale).to(torch.bfloat16)
        self.mass = torch.rand((len(lens), H, self.mb), generator=g)

    @property
    def sl(self):
        return torch.tensor(self.lens, dtype=torch.int32)

    def select(self, positions, fill=1.0):
        """16 slots per query: a random subset of its causal blocks, some slots empty, in any order."""
        sel = torch.full((len(positions), 16), -1, dtype=torch.int32)
        for i, p in enumerate(positions):
            nb = p // BLOCK + 1 if p >= 0 else 0
            k = min(16, nb, max(0, int(round(fill * 16))))
            pick = torch.randperm(nb, generator=self.g)[:k] if nb else torch.empty(0, dtype=torch.long)
            at = torch.randperm(16, generator=self.g)[:k]
            sel[i, at] = pick.to(torch.int32)
        return sel

    def want(self, i, b, p, blocks, scale):
        blocks = [j for j in blocks if j >= 0]
        pages = [int(self.table[b, j]) for j in blocks]
        return ref.attend(self.q[i], self.k, self.v, self.ks, self.vs, pages, blocks, p, scale) + (blocks,)

    def gpu(self, dev):
        return to(dev, self.q, self.k, self.v, self.ks, self.vs, self.table, self.sl)


def check_rows(case, out, mass, rows, scale=128 ** -0.5, many=False):
    """rows: (query, sequence, position, blocks).  mass: the GPU's totals, or None."""
    out = out.float().cpu().double()
    total = case.mass.double().clone()
    bound = torch.zeros_like(total)
    count = {}
    for i, b, p, blocks in rows:
        o, w, mag, vmax, used = case.want(i, b, p, blocks, scale)
        err = (out[i] - o).abs()
        lim = ref.out_bound(o, mag, vmax, many)
        assert (err <= lim).all(), (i, float((err / lim).max()))
        for x, j in enumerate(used):
            total[b, :, j] += w[:, x]
            bound[b, :, j] += ref.mass_bound(total[b, :, j], mag)
        count[b] = count.get(b, 0) + 1
    if mass is not None:
        err = (mass.cpu().double() - total).abs()
        assert (err <= bound).all(), float((err - bound).max())   # untouched totals: equal


LENS = [[1], [0, 31, 32, 33], [512, 513, 511, 2000], [129, 0, 4096, 7, 700]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H", [1, 10, 12])
@pytest.mark.parametrize("odd_scale", [False, True])
def test_sparse_decode_attention(uocr, cuda_device, lens, H, odd_scale):
    c = Case(lens, H, seed=len(lens) * 100 + H, odd_scale=odd_scale)
    pos = [x - 1 for x in lens]
    sel = c.select(pos)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), mass=mass)
    check_rows(c, out, mass, [(i, i, pos[i], sel[i].tolist()) for i in range(len(lens))])
    again = c.mass.to(cuda_device)
    out2 = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), mass=again)
    assert torch.equal(out, out2) and torch.equal(mass, again)
    assert torch.equal(out, uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device)))


@pytest.mark.parametrize("fill", [0.0, 0.2, 1.0])
def test_sparse_many_queries_per_sequence_and_scale(uocr, cuda_device, fill):
    c = Case([700, 90, 2100], 5, seed=7, n_q=9)
    seq = [0, 0, 1, 2, 2, 2, 1, 0, 2]
    pos = [699, 0, 89, 31, 32, 2099, 5, 340, 1000]
    sel = c.select(pos, fill)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), torch.tensor(seq, dtype=torch.int32, device=cuda_device),
                               torch.tensor(pos, dtype=torch.int32, device=cuda_device), scale=0.3)
    check_rows(c, out, None, [(i, seq[i], pos[i], sel[i].tolist()) for i in range(9)], scale=0.3)


def test_sparse_duplicate_slots_count_twice(uocr, cuda_device):
    c = Case([300], 3, seed=8)
    sel = torch.tensor([[2, 9, 2, -1, 5, 2, 9, -1, -1, -1, 0, -1, -1, -1, -1, 5]], dtype=torch.int32)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), mass=mass)
    check_rows(c, out, mass, [(0, 0, 299, sel[0].tolist())])


@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 1e-3, 30.0, 1e20])
def test_sparse_query_magnitudes(uocr, cuda_device, q_scale):
    """Queries far outside fp16's range: a flat softmax for tiny ones, one token's value for huge ones."""
    c = Case([400, 64], 4, seed=9, q_scale=q_scale)
    sel = c.select([399, 63])
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device)).float().cpu().double()
    for i, p in enumerate((399, 63)):
        o, w, mag, vmax, used = c.want(i, i, p, sel[i].tolist(), 128 ** -0.5)
        if q_scale <= 30:
            assert ((out[i] - o).abs() <= ref.out_bound(o, mag, vmax)).all()
        else:
            assert torch.isfinite(out[i]).all() and (out[i].abs() <= vmax[:, None] * (1 + 2.0 ** -8)).all()


def test_sparse_not_finite_query_stays_its_own(uocr, cuda_device):
    c = Case([200, 300, 100], 2, seed=10)
    c.q[1, 0, 5] = math.nan
    c.q[1, 1, 7] = math.inf
    sel = c.select([199, 299, 99])
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), mass=mass)
    check_rows(c, out, None, [(i, i, p, sel[i].tolist()) for i, p in ((0, 199), (2, 99))])
    assert torch.isnan(out[1, 0].float()).all()
    assert torch.isfinite(mass).all() and torch.equal(mass[1, 0].cpu(), c.mass[1, 0])


def test_sparse_device_errors(uocr, cuda_device):
    c = Case([200, 300, 100, 50], 2, seed=11)
    sel = c.select([199, 299, 99, 49])
    sel[0, :] = torch.tensor([7] + [-1] * 15)            # block 7 of 7 is past the end
    c.table[1, int(sel[1][sel[1] >= 0][0])] = 10 ** 6    # outside the pool
    bad = int(sel[1][sel[1] >= 0][0])
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    sl[3] = c.mb * BLOCK + 1
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), mass=mass, dev_err=err)
    assert int(err) == uocr.DEVERR_SEL | uocr.DEVERR_PAGE | uocr.DEVERR_POS
    assert (out[0].float() == 0).all() and (out[3].float() == 0).all()
    left = [j for j in sel[1].tolist() if j >= 0 and j != bad]
    check_rows(c, out, mass, [(1, 1, 299, left), (2, 2, 99, sel[2].tolist())])


@pytest.mark.parametrize("H", [3, 40])       # few rows: a query at a time; many: block by block
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-3])
def test_any_finite_scale(uocr, cuda_device, scale, H):
    """A negative scale turns the order of the scores round, 0 makes them all equal (also next to tokens that are
    behind the query)."""
    n, total = 20, 150
    c = Case([total], H, seed=17, n_q=n)
    pos = list(range(total - n, total))
    sel = torch.full((n, 16), -1, dtype=torch.int32)
    sel[:, 3:8] = torch.arange(5)
    sel[:14, 7] = torch.tensor([4 if p >= 128 else -1 for p in pos[:14]], dtype=torch.int32)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    qp, se = torch.tensor(pos, dtype=torch.int32, device=cuda_device), sel.to(cuda_device)
    rows = [(i, 0, pos[i], sel[i].tolist()) for i in range(n)]
    one = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, se, torch.zeros(n, dtype=torch.int32, device=cuda_device), qp, scale=scale)
    check_rows(c, one, None, rows, scale=scale)
    mass = c.mass.to(cuda_device)
    many = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 0, qp, se, scale=scale, mass=mass)
    check_rows(c, many, mass, rows, scale=scale, many=True)


@pytest.mark.parametrize("H", [64])
def test_most_heads(uocr, cuda_device, H):
    c = Case([70, 700], H, seed=18)
    sel = c.select([69, 699])
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    rows = [(i, i, c.lens[i] - 1, sel[i].tolist()) for i in range(2)]
    mass = c.mass.to(cuda_device)
    check_rows(c, uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), mass=mass), mass, rows)
    out = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl)
    check_rows(c, out, None, [(i, i, c.lens[i] - 1, list(range(-(-c.lens[i] // 32)))) for i in range(2)])
    out = uocr.sparse_attn_seq_kv8(q[1:], k, v, ks, vs, bt, sl, 1, torch.tensor([699], dtype=torch.int32, device=cuda_device),
                                   sel[1:].to(cuda_device))
    c.q = c.q[1:]
    check_rows(c, out, None, [(0, 1, 699, sel[1].tolist())], many=True)


def test_pools_past_32_bit_offsets(uocr, cuda_device):
    """Pages whose tiles lie behind 4 GiB: read by every form, written by the append."""
    H, P, total = 10, 110000, 300
    c = Case([total], H, seed=19)
    used = c.table[0, :10].long()
    far = torch.arange(P - 10, P)
    codes = [torch.zeros(P * H * 4096, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    scales = [torch.ones((P, H), device=cuda_device) for _ in range(2)]
    k8, v8 = [x.view(torch.float8_e4m3fn).view(P, H, 32, 128) for x in codes]
    for dst, src in ((codes[0], c.k), (codes[1], c.v)):
        dst.view(P, H, 32, 128)[P - 10:] = src.view(torch.uint8)[used].to(cuda_device)
    scales[0][P - 10:], scales[1][P - 10:] = c.ks[used].to(cuda_device), c.vs[used].to(cuda_device)
    bt = far.to(torch.int32)[None].to(cuda_device).contiguous()
    q, sl = c.q.to(cuda_device), c.sl.to(cuda_device)
    sel = torch.full((1, 16), -1, dtype=torch.int32)
    sel[0, :10] = torch.arange(10)
    pos = torch.tensor([total - 1], dtype=torch.int32, device=cuda_device)
    rows = [(0, 0, total - 1, list(range(10)))]
    check_rows(c, uocr.sparse_attn_kv8(q, k8, v8, *scales, bt, sl, sel.to(cuda_device)), None, rows)
    check_rows(c, uocr.dense_decode_kv8(q, k8, v8, *scales, bt, sl), None, rows)
    for n in (1, 80):    # a query at a time, and block by block
        out = uocr.sparse_attn_seq_kv8(q.expand(n, -1, -1).contiguous(), k8, v8, *scales, bt, sl, 0, pos.expand(n).contiguous(),
                                       sel.to(cuda_device).expand(n, -1).contiguous())
        check_rows(c, out, None, rows, many=True)
        assert torch.equal(out, out[:1].expand(n, -1, -1))
    g = torch.Generator().manual_seed(1)
    for n in (1, 40):    # both of the append's forms
        rnd = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16)  # noqa: E731
        s = {"q": rnd(n, H, 128), "idx_q": rnd(n, 128), "k_new": rnd(n, H, 128), "v_new": rnd(n, H, 128), "idx_k_new": rnd(n, 128),
             "tok": torch.arange(n, dtype=torch.int32), "page": torch.zeros(n, dtype=torch.int32), "idx_k": torch.zeros((10, 32, 128), dtype=torch.bfloat16)}
        for name, x, sc in (("k", k8, scales[0]), ("v", v8, scales[1])):
            s[name], s[name + "_scale"] = x[P - 10:].cpu(), sc[P - 10:].cpu()
        want = ref.append(s, [0, n], [total], torch.arange(10, dtype=torch.int32)[None])
        ik = torch.zeros((P, 32, 128), dtype=torch.bfloat16, device=cuda_device)
        d = {x: s[x].to(cuda_device) for x in ("q", "idx_q", "k_new", "v_new", "idx_k_new", "tok", "page")}
        uocr.rope_append_kv8(*d.values(), bt, sl, k8, v8, *scales, ik, torch.tensor([0, n], dtype=torch.int32, device=cuda_device))
        for name, x, sc in (("k", k8, scales[0]), ("v", v8, scales[1])):
            assert same_codes(x[P - 10:].cpu(), want[name])
            assert np.array_equal(sc[P - 10:].cpu().double().numpy(), want[name + "_scale"])
            assert (x[:1000].view(torch.uint8) == 0).all() and (sc[:P - 10] == 1).all()


@pytest.mark.parametrize("lens,ref_blocks", [([1], None), ([0, 31, 32, 33], None), ([2000, 513, 5000], None), ([2000, 513, 5000, 0, 90], 3),
                                             ([1000, 64], 0), ([700, 3000], 22), ([9001], 10 ** 6)])
@pytest.mark.parametrize("H", [1, 10])
def test_dense_decode(uocr, cuda_device, lens, ref_blocks, H):
    c = Case(lens, H, seed=sum(lens) + H, odd_scale=H == 1)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, ref_blocks=ref_blocks, mass=mass)
    rows = []
    for b, x in enumerate(lens):
        nb = -(-x // BLOCK)
        rb = c.mb if ref_blocks is None else ref_blocks
        rows.append((b, b, x - 1, [j for j in range(nb) if j < rb or j >= nb - 4]))
    check_rows(c, out, mass, rows)
    again = c.mass.to(cuda_device)
    ws = torch.full((uocr.dense_kv8_workspace_bytes(len(lens), H, c.mb),), 0xFF, dtype=torch.uint8, device=cuda_device)
    out2 = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, ref_blocks=ref_blocks, mass=again, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(mass, again)       # whatever the workspace held
    assert torch.equal(out, uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, ref_blocks=ref_blocks))


def test_dense_bad_pages_and_lengths(uocr, cuda_device):
    c = Case([900, 400, 50], 3, seed=12)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    bt[0, 5] = -1
    bt[0, 28] = 1 << 30
    sl[1] = c.mb * BLOCK + 5
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, mass=mass, dev_err=err)
    assert int(err) == uocr.DEVERR_PAGE | uocr.DEVERR_POS
    assert (out[1].float() == 0).all()
    check_rows(c, out, mass, [(0, 0, 899, [j for j in range(29) if j not in (5, 28)]), (2, 2, 49, [0, 1])])


def test_a_block_of_nan_scale_or_all_minus_inf(uocr, cuda_device):
    """A page whose scale is 0 counts as zeros; an infinite score takes the row to NaN, as the formula does."""
    c = Case([300], 2, seed=13)
    c.vs[int(c.table[0, 3])] = 0.0
    c.ks[int(c.table[0, 4])] = 0.0
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    out = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl)
    check_rows(c, out, None, [(0, 0, 299, list(range(10)))])


@pytest.mark.parametrize("total,n,H", [(1, 1, 1), (33, 33, 3), (700, 1, 10), (700, 17, 10), (1300, 333, 4), (4100, 130, 12)])
@pytest.mark.parametrize("order", ["chunk", "any"])
def test_many_queries_of_a_sequence(uocr, cuda_device, total, n, H, order):
    c = Case([total, 64], H, seed=total + n, n_q=n, odd_scale=order == "any")
    pos = list(range(total - n, total))
    if order == "any":
        pos = torch.randint(0, total, (n,), generator=c.g).tolist()
    sel = c.select(pos, 1.0 if order == "chunk" else 0.6)
    if order == "chunk":     # the real shape: the 4 local blocks among them
        for i, p in enumerate(pos):
            nb = p // BLOCK + 1
            sel[i, 12:] = -1
            sel[i] = torch.where((sel[i] >= nb - 4), -1, sel[i])
            sel[i, 12:] = torch.tensor([j if j >= 0 else -1 for j in range(nb - 4, nb)], dtype=torch.int32)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    qp, se = torch.tensor(pos, dtype=torch.int32, device=cuda_device), sel.to(cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 0, qp, se, mass=mass)
    check_rows(c, out, mass, [(i, 0, pos[i], sel[i].tolist()) for i in range(n)], many=True)
    again = c.mass.to(cuda_device)
    ws = torch.full((uocr.sparse_attn_seq_kv8_workspace_bytes(n, H, c.mb),), 0xFF, dtype=torch.uint8, device=cuda_device)
    out2 = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 0, qp, se, mass=again, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(mass, again)
    # and the per-query form agrees within both bounds
    one = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, se, torch.zeros(n, dtype=torch.int32, device=cuda_device), qp)
    check_rows(c, one, None, [(i, 0, pos[i], sel[i].tolist()) for i in range(n)])


@pytest.mark.parametrize("H", [2, 30])
def test_many_queries_later_nan_does_not_reach_earlier_ones(uocr, cuda_device, H):
    """A token whose value is NaN is behind some queries of its block: theirs stay finite."""
    c = Case([160], H, seed=14, n_q=32)
    pos = list(range(128, 160))
    c.v.view(torch.uint8)[int(c.table[0, 4]), 1, 20, 3] = 0xFF
    sel = torch.full((32, 16), -1, dtype=torch.int32)
    sel[:, :3] = torch.tensor([0, 2, 4])
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    out = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 0, torch.tensor(pos, dtype=torch.int32, device=cuda_device), sel.to(cuda_device))
    check_rows(c, out, None, [(i, 0, pos[i], [0, 2, 4]) for i in range(20)], many=True)
    o = out.float().cpu()
    assert torch.isnan(o[20:, 1, 3]).all()
    o[20:, 1, 3] = 0
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("times", [1, 80])
def test_many_queries_bad_slots_positions_and_pages(uocr, cuda_device, times):
    c = Case([640], 2, seed=15, n_q=6 * times)
    pos = [639, 700, -1, 100, 5, 300] * times
    sel = c.select([639, 639, 639, 100, 5, 300] * times, 0.5)
    c.table[0, 2] = -5
    for x in range(times):
        sel[6 * x + 3] = torch.tensor([19, 3, 1, 3, -7] + [-1] * 11)       # 19: not causal; 3 twice
        sel[6 * x + 5] = torch.tensor([2, 4] + [-1] * 14)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 0, torch.tensor(pos, dtype=torch.int32, device=cuda_device), sel.to(cuda_device),
                                   mass=mass, dev_err=err)
    assert int(err) == uocr.DEVERR_SEL | uocr.DEVERR_PAGE | uocr.DEVERR_POS
    assert all((out[6 * x + 1:6 * x + 3].float() == 0).all() for x in range(times))
    fine = lambda i: [j for j in sel[i].tolist() if 0 <= j <= pos[i] // BLOCK and j != 2]  # noqa: E731
    check_rows(c, out, mass, [(6 * x + i, 0, pos[i], fine(6 * x + i)) for x in range(times) for i in (0, 3, 4, 5)], many=True)


@pytest.mark.parametrize("empty", [-2, -1, -3, -(1 << 31)])
def test_any_negative_slot_is_empty(uocr, cuda_device, empty):
    """Slots below 0 in every place of the selection, of queries with at most 16 causal blocks and with more: through
    the decode form and through both forms of many queries."""
    H, lens = 10, [200, 1000]
    for b, total in enumerate(lens):
        for n in (5, 100):      # n * H up to 5 a SM: a query at a time; more: block by block
            c = Case(lens, H, seed=90 + b, n_q=n)
            pos = [total - 1 - (7 * i) % 130 for i in range(n)]
            sel = torch.full((n, 16), empty, dtype=torch.int32)
            for i, p in enumerate(pos):
                nb = p // BLOCK + 1
                if i % 5 == 1:                                     # 12 .. 15 empty
                    sel[i, :3] = torch.tensor([nb - 1, 0, nb // 2])
                elif i % 5 == 2:                                   # below 12 empty
                    sel[i, 12:14] = torch.tensor([nb - 1, 0])
                elif i % 5 == 3:
                    sel[i, ::3] = torch.tensor([nb - 1, 0, nb // 2, empty, 1, empty])
                elif i % 5 == 4:
                    sel[i, 5] = nb - 1                             # (i % 5 == 0: nothing is selected)
            q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
            qp, se = torch.tensor(pos, dtype=torch.int32, device=cuda_device), sel.to(cuda_device)
            rows = [(i, b, pos[i], sel[i].tolist()) for i in range(n)]
            mass = c.mass.to(cuda_device)
            check_rows(c, uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, b, qp, se, mass=mass), mass, rows, many=True)
            seq = torch.full((n,), b, dtype=torch.int32, device=cuda_device)
            check_rows(c, uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, se, seq, qp), None, rows)
    c = Case(lens, H, seed=92)  # a query per sequence, with totals
    sel = torch.full((2, 16), empty, dtype=torch.int32)
    sel[0, 2], sel[1, 13] = 1, 30
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel.to(cuda_device), mass=mass)
    check_rows(c, out, mass, [(i, i, lens[i] - 1, sel[i].tolist()) for i in range(2)])


def every_form(uocr, dev, c, n, scale):
    """The attention of case c's n queries (rows of sequence 0, in blocks of its tokens from the last one back) by every
    form: yields name, output, totals, rows and whether it is the block by block one."""
    total = c.lens[0]
    pos = [total - 1 - 5 * (i % 40) for i in range(n)]
    nb = -(-total // BLOCK)
    assert nb <= 16
    sel = torch.full((n, 16), -1, dtype=torch.int32)
    for i, p in enumerate(pos):
        sel[i, :p // BLOCK + 1] = torch.arange(p // BLOCK + 1)
    q, k, v, ks, vs, bt, sl = c.gpu(dev)
    qp, se, seq = torch.tensor(pos, dtype=torch.int32, device=dev), sel.to(dev), torch.zeros(n, dtype=torch.int32, device=dev)
    rows = [(i, 0, pos[i], sel[i].tolist()) for i in range(n)]
    yield "sparse", uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, se, seq, qp, scale=scale), None, rows, False
    for m in (5, n):
        mass = c.mass.to(dev)
        yield f"seq {m}", uocr.sparse_attn_seq_kv8(q[:m], k, v, ks, vs, bt, sl, 0, qp[:m], se[:m], scale=scale, mass=mass), mass, rows[:m], m == n
    mass = c.mass.to(dev)
    yield "one", uocr.sparse_attn_kv8(q[:1], k, v, ks, vs, bt, sl, se[:1], scale=scale, mass=mass), mass, rows[:1], False
    if scale is None or abs(scale - 128 ** -0.5) < 1e-9:
        mass = c.mass.to(dev)
        yield "dense", uocr.dense_decode_kv8(q[:1], k, v, ks, vs, bt, sl, mass=mass), mass, rows[:1], False


@pytest.mark.parametrize("q_scale,k_factor,scale", [(1e37, 2.0 ** -124, 128 ** -0.5),    # the row's unit times a product leaves fp32
                                                    (1e-34, 2.0 ** 112, 128 ** -0.5),
                                                    (1.0, -1.0, 128 ** -0.5), (1.0, -2.0 ** -3, -0.3),
                                                    (0.0, 2.0 ** 129, 128 ** -0.5),      # products of 0 under scales near fp32's end
                                                    (0.0, -2.0 ** 129, 100.0), (0.0, 2.0 ** 120, -1e6),
                                                    (1e-30, 2.0 ** 129, 2.0 ** -30),
                                                    (1.0, 1.0, 0.0)])
def test_any_finite_key_scale_in_every_form(uocr, cuda_device, q_scale, k_factor, scale):
    c = Case([450], 10, seed=94, n_q=100, q_scale=q_scale)
    c.ks = (c.ks.double() / c.ks.max() * 2.0 ** -4 * k_factor).float()     # largest: 2^-4 k_factor
    assert torch.isfinite(c.ks).all()
    for name, out, mass, rows, many in every_form(uocr, cuda_device, c, 100, scale):
        check_rows(c, out, mass, rows, scale=scale, many=many)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("q_scale", [0.0, 1.0])
def test_a_scale_that_is_not_finite_stays_with_its_rows(uocr, cuda_device, bad, which, q_scale):
    """Head 3 of block 12 has such a scale: the rows that attend it are not finite (NaN for K) in that head, and theirs
    alone; the K scale's weights add nothing, the V scale's are those of a finite one."""
    c = Case([450], 10, seed=95, n_q=100, q_scale=q_scale)
    page = int(c.table[0, 12])
    plain = c.ks.clone(), c.vs.clone()
    for name, out, mass, rows, many in every_form(uocr, cuda_device, c, 100, None):
        (c.ks if which == "k" else c.vs)[page, 3] = bad
        again = dict((x[0], x) for x in every_form(uocr, cuda_device, c, 100, None))[name]
        c.ks, c.vs = plain[0].clone(), plain[1].clone()
        hit = torch.tensor([p // BLOCK >= 12 for _, _, p, _ in rows])
        got = again[1].float().cpu()
        assert torch.isnan(got[hit][:, 3]).all() if which == "k" else not torch.isfinite(got[hit][:, 3]).any(), name
        same = torch.ones_like(got, dtype=torch.bool)
        same[hit, 3] = False
        assert torch.equal(got[same], out.float().cpu()[same]), name
        if mass is not None:
            if which == "v":
                assert torch.equal(mass, again[2]), name
            else:
                heads = [h for h in range(10) if h != 3]
                assert torch.equal(mass[:, heads], again[2][:, heads]) and torch.isfinite(again[2]).all(), name
                rest = c.mass.clone()
                clean = [(i, b, p, x) for i, b, p, x in rows if p // BLOCK < 12]
                for i, b, p, x in clean:
                    _, w, _, _, used = c.want(i, b, p, x, 128 ** -0.5)
                    for y, j in enumerate(used):
                        rest[b, 3, j] += w[3, y]
                assert ((again[2][:, 3].cpu() - rest[:, 3]).abs() <= 1e-4 * rest[:, 3].abs() + 1e-30).all(), name


@pytest.mark.parametrize("form", ["sparse", "seq", "dense"])
def test_light_blocks_under_large_value_scales(uocr, cuda_device, form):
    """A block whose weights are 2^-23 of another's and whose value scale is 2^23 of the other's counts as much: its
    weights keep their bits, whichever of the two a warp meets first."""
    H, n, total = 10, 100, 32 * 32
    c = Case([total] * (n if form != "seq" else 1), H, seed=96, n_q=n)
    c.ks[:] = 2.0 ** -30
    heavy = torch.zeros(c.k.shape[0], dtype=torch.bool)
    heavy[c.table[:, [3, 17, 24]].long().flatten()] = True
    c.q[:] = c.q.abs() + 1
    c.k.view(torch.uint8)[heavy] = torch.tensor([1.0]).to(ref.E4M3).view(torch.uint8)      # q . k = sum of q, alike for a block's tokens
    per = c.q.double().sum(-1) * 128 ** -0.5
    c.ks[heavy] = float(23 * math.log(2) / per.mean())
    c.vs[heavy] *= 2.0 ** -23
    c.v.view(torch.uint8)[:] &= 0x7F      # of one sign, so that a weight's error shows
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    blocks = [0, 3, 5, 8, 9, 11, 12, 13, 16, 17, 20, 21, 23, 24, 27, 31]
    se = torch.tensor([blocks] * n, dtype=torch.int32, device=cuda_device)
    if form == "sparse":         # 1000 pairs: a warp attends four blocks
        out = uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, se)
    elif form == "seq":
        out = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 0, torch.full((n,), total - 1, dtype=torch.int32, device=cuda_device), se)
    else:
        out, blocks = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl), list(range(32))
    out = out.float().cpu().double()
    for i in range(0, n, 7):
        o, w, mag, vmax, _ = c.want(i, i if form != "seq" else 0, total - 1, blocks, 128 ** -0.5)
        # what the light blocks' values add, with the weights' error (2^-22 of a weight in two fp16 numbers; 2^-11 in one
        # and as much of a partial output; ref.weight_bound for the fp32 part), bf16's half step
        light = torch.tensor([not bool(heavy[int(c.table[i if form != "seq" else 0, j])]) for j in blocks])
        size = w[:, light].sum(-1) * vmax + 2.0 ** -23 * vmax
        lim = o.abs() * 2.0 ** -8 + (size * (ref.weight_bound(mag) + (2.0 ** -10 if form == "seq" else 2.0 ** -22)))[:, None]
        assert ((out[i] - o).abs() <= lim).all(), (i, float(((out[i] - o).abs() / lim).max()))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_stays_its_own_in_every_form(uocr, cuda_device, bad):
    """Its row and head is NaN, its weights add nothing; every other row, head and total is what it is without it."""
    c = Case([450], 10, seed=97, n_q=100)
    fine = c.q.clone()
    for name, out, mass, rows, many in every_form(uocr, cuda_device, c, 100, None):
        hit = torch.zeros((len(rows), 10), dtype=torch.bool)
        for i, h in ((0, 3), (2, 9), (17, 0)):
            if i < len(rows):
                c.q[i, h, 11 * h + 5], hit[i, h] = bad, True
        again = dict((x[0], x) for x in every_form(uocr, cuda_device, c, 100, None))[name]
        c.q = fine.clone()
        got = again[1].float().cpu()
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], out.float().cpu()[~hit]), name
        if mass is not None:
            total = c.mass.double()
            for i, b, p, x in rows:
                _, w, _, _, used = c.want(i, b, p, x, 128 ** -0.5)
                for y, j in enumerate(used):
                    total[b, :, j] += torch.where(hit[i], 0.0, w[:, y])
            assert ((again[2].cpu().double() - total).abs() <= 1e-4 * total + 1e-30).all(), name


@pytest.mark.parametrize("n", [5, 100])      # a query at a time; block by block
@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 1e-3, 30.0, 1e7, 1e8, 1e9, 1e20])
def test_many_queries_of_any_magnitude(uocr, cuda_device, n, q_scale):
    """From a flat softmax to scores far past 2^31: where the highest score leads by more than the products' error
    (ref.weight_bound: 2^-18 of the sum of magnitudes each) and 2^10, the output is that token's value."""
    H, total, scale = 10, 700, 128 ** -0.5
    c = Case([total], H, seed=93, n_q=n, q_scale=q_scale)
    pos = [total - 1 - 3 * (i % 70) for i in range(n)]
    sel = c.select(pos)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    mass = c.mass.to(cuda_device)
    out = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 0, torch.tensor(pos, dtype=torch.int32, device=cuda_device), sel.to(cuda_device), mass=mass)
    if q_scale <= 30:
        check_rows(c, out, mass, [(i, 0, pos[i], sel[i].tolist()) for i in range(n)], many=True)
        return
    assert torch.isfinite(mass).all() and abs(float(mass.sum() - c.mass.sum().to(cuda_device)) - n * H) < 1e-4 * float(mass.sum())
    got, clear = out.float().cpu().double(), 0
    for i, p in enumerate(pos):
        blocks = [j for j in sel[i].tolist() if j >= 0]
        pg = c.table[0, blocks].long()
        see = (torch.tensor(blocks)[:, None] * BLOCK + torch.arange(BLOCK) <= p).reshape(-1)
        kk, vv = ((ref.values(x[pg]) * s[pg].double()[:, :, None, None]).transpose(0, 1).reshape(H, -1, 128)[:, see] for x, s in ((c.k, c.ks), (c.v, c.vs)))
        z = torch.einsum("htd,hd->ht", kk, c.q[i].double()) * scale
        err = (kk.abs() * c.q[i].double().abs()[:, None]).sum(-1).amax(dim=1) * scale * 2.0 ** -18
        top, at = z.topk(2, dim=1)
        lead = top[:, 0] - top[:, 1] > 2 * err + 2 ** 10
        want = vv[torch.arange(H), at[:, 0]]
        assert torch.isfinite(got[i]).all()
        assert ((got[i] - want).abs() <= want.abs() * 2.0 ** -8 + 1e-38)[lead].all()
        clear += int(lead.sum())
    assert clear > 0.9 * n * H


def test_many_queries_wait_timeout_is_flagged_and_recovers(uocr, cuda_device):
    """The waits for the keys give up at once: every block is dropped and flagged, the copies are waited
    for before their shared memory goes, and the next call is whole."""
    case = Case([32 * 200], 10, seed=71, n_q=100)
    positions = torch.arange(6000, 6100, dtype=torch.int32)
    sel = case.select(positions.tolist())
    q, k, v, ks, vs, table, sl = case.gpu(cuda_device)
    pos, s = to(cuda_device, positions, sel)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)

    def run():
        (mass,) = to(cuda_device, case.mass)
        out = uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, table, sl, 0, pos, s, mass=mass, dev_err=err)
        torch.cuda.synchronize()
        return out, mass

    limit = uocr.lib.uocr_test_first_wait_limit_ns
    limit.argtypes, limit.restype = [ctypes.c_longlong], None
    limit(0)
    try:
        out, mass = run()
    finally:
        limit(-1)
    assert int(err.item()) & uocr.DEVERR_TIMEOUT
    assert (out == 0).all() and torch.equal(mass.cpu(), case.mass)
    err.zero_()
    out, mass = run()
    assert int(err.item()) == 0
    rows = [(i, 0, int(positions[i]), sel[i].tolist()) for i in range(100)]
    check_rows(case, out, mass, rows, many=True)


# ------------------------------------------------------------------------------------------ append
def append_state(seed, H, lens, new, extra_rows=0, spare=3):
    g = torch.Generator().manual_seed(seed)
    mb = max(1, max(-(-x // BLOCK) for x in lens))
    table, pages = ref.make_table(g, lens, mb, spare)
    n = sum(new) + extra_rows
    s = {}
    s["k"], s["k_scale"] = ref.make_pool(g, pages, H)
    s["v"], s["v_scale"] = ref.make_pool(g, pages, H)
    for name, shape in (("q", (n, H, 128)), ("idx_q", (n, 128)), ("k_new", (n, H, 128)), ("v_new", (n, H, 128)), ("idx_k_new", (n, 128)),
                        ("idx_k", (pages, BLOCK, 128))):
        s[name] = torch.randn(shape, generator=g).to(torch.bfloat16)
    for name in ("k_new", "v_new"):      # some raise their page's scale, some do not
        s[name] *= torch.exp(1.2 * torch.randn((n, H, 1), generator=g)).to(torch.bfloat16)
    s["tok"] = torch.randint(0, 120000, (n,), generator=g, dtype=torch.int32)
    s["page"] = torch.randint(-3, 50, (n,), generator=g, dtype=torch.int32)
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    return s, table, starts, n


def run_append(uocr, dev, s, table, lens, starts, in_place=False, dev_err=None, null_start=False):
    d = {k: v.clone().to(dev) for k, v in s.items()}
    bt, sl = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    q_out = None if in_place else torch.full_like(d["q"], 7.0)
    i_out = None if in_place else torch.full_like(d["idx_q"], 7.0)
    st = None if null_start else torch.tensor(starts, dtype=torch.int32, device=dev)
    q, i = uocr.rope_append_kv8(d["q"], d["idx_q"], d["k_new"], d["v_new"], d["idx_k_new"], d["tok"], d["page"], bt, sl, d["k"], d["v"],
                                d["k_scale"], d["v_scale"], d["idx_k"], st, q_out=q_out, idx_q_out=i_out, dev_err=dev_err)
    torch.cuda.synchronize()
    assert (q.data_ptr() == d["q"].data_ptr()) == in_place
    return q, i, {k: d[k].cpu() for k in ("k", "v", "k_scale", "v_scale", "idx_k")}


def same_codes(a, b):
    """Codes equal, NaN in either sign."""
    a, b = a.view(torch.uint8).numpy(), b
    return bool(((a == b) | ((a & 127 == 127) & (b & 127 == 127))).all())


def check_append(s, got, want, old_q):
    q, i, caches = got
    for name in ("k", "v"):
        assert same_codes(caches[name], want[name]), name
        assert np.array_equal(caches[name + "_scale"].double().numpy(), want[name + "_scale"]), name
    for t, w, old in ((q, want["q"], old_q[0]), (i, want["idx_q"], old_q[1])):
        t = t.float().cpu().double().numpy()
        put = np.isfinite(w)
        assert (np.abs(t - w)[put] <= np.abs(w[put]) * 2.0 ** -8 + 1e-38).all()
        assert np.array_equal(t[~put], old.double().numpy()[~put])            # rows that belong to no sequence
    k, w = caches["idx_k"].double().numpy(), want["idx_k"]
    assert (np.abs(k - w) <= np.where(want["wrote"][..., None], np.abs(w) * 2.0 ** -8 + 1e-38, 0)).all()


@pytest.mark.parametrize("lens,new", [([1], [1]), ([32, 33, 64, 5], [1, 1, 1, 1]), ([100], [100]), ([77, 5, 200], [40, 5, 70]),
                                      ([300, 31, 64, 96, 1], [257, 0, 32, 33, 1]), ([33, 65], [2, 34]), ([700], [1])])
@pytest.mark.parametrize("H", [1, 10])
def test_append(uocr, cuda_device, lens, new, H):
    s, table, starts, n = append_state(sum(lens) + H, H, lens, new, extra_rows=2)
    want = ref.append(s, starts, lens, table)
    got = run_append(uocr, cuda_device, s, table, lens, starts)
    check_append(s, got, want, (torch.full_like(s["q"], 7.0), torch.full_like(s["idx_q"], 7.0)))
    place = run_append(uocr, cuda_device, s, table, lens, starts, in_place=True)
    check_append(s, place, want, (s["q"], s["idx_q"]))
    if new == [1] * len(lens):
        s2 = {k: (v[:n - 2] if v.shape[0] == n and k not in ("k", "v", "k_scale", "v_scale", "idx_k") else v) for k, v in s.items()}
        one = run_append(uocr, cuda_device, s2, table, lens, starts, null_start=True)
        for k in ("k", "v"):
            assert same_codes(one[2][k], want[k])


def test_append_is_the_same_in_any_chunks(uocr, cuda_device):
    """One chunk of 90 tokens, or the same 90 in calls of one: equal values wherever the scale did not need a second
    rounding, and equal scales."""
    H, lens = 3, [90]
    s, table, starts, n = append_state(5, H, lens, [90])
    _, _, whole = run_append(uocr, cuda_device, s, table, lens, starts)
    dev = cuda_device
    d = {k: v.clone().to(dev) for k, v in s.items()}
    bt = table.to(dev)
    for i in range(90):
        sl = torch.tensor([i + 1], dtype=torch.int32, device=dev)
        uocr.rope_append_kv8(*[d[x][i:i + 1].clone() for x in ("q", "idx_q", "k_new", "v_new", "idx_k_new", "tok", "page")], bt, sl,
                             d["k"], d["v"], d["k_scale"], d["v_scale"], d["idx_k"])
    for x in "kv":
        used = [int(p) for p in table[0]]
        a, b = whole[x + "_scale"][used], d[x + "_scale"].cpu()[used]
        assert torch.equal(a, b)
        va, vb = ref.values(whole[x])[used], ref.values(d[x])[used]
        rows = torch.arange(3 * BLOCK).reshape(3, 1, BLOCK, 1) < 90
        # below e4m3's normal range (2^-6) a code may have been rounded twice: by at most a step of 2^-9
        diff = torch.where(rows, (va - vb).abs(), 0.0)
        assert (diff <= torch.where(va.abs() < 2.0 ** -5, 2.0 ** -9, 0.0)).all()
    assert torch.equal(whole["idx_k"], d["idx_k"].cpu())


def bf16_rounded(x):
    """64-bit values to the nearest bf16 (ties to even, past the last one to infinity), and how far each is from a
    midpoint."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x)
    a = np.where(fine, np.abs(x), 0.0)
    step = np.ldexp(1.0, np.maximum(np.frexp(a)[1] - 8, -133))
    y = np.rint(a / step) * step
    gap = np.abs(np.abs(a / step - np.floor(a / step)) - 0.5) * step
    y = np.where(y > 3.3895314e38, np.inf, y)
    return np.where(fine, np.copysign(y, x), x), gap


def test_append_rounds_once_in_both_kernels(uocr, cuda_device):
    """The same tokens as 6 a sequence (the kernel for few) and beside a longer sequence (the one for many): equal
    queries, indexer vectors, codes and scales, and each the 64-bit rotation rounded once to bf16."""
    H, B = 10, 160
    lens, new = [6 + (5 * b) % 70 for b in range(B)] + [40], [6] * B + [40]
    s, table, starts, n = append_state(80, H, lens, new)
    few = {x: (v[:6 * B] if v.shape[0] == n else v) for x, v in s.items()}
    got = [run_append(uocr, cuda_device, few, table[:B], lens[:B], starts[:B + 1]), run_append(uocr, cuda_device, s, table, lens, starts)]
    pages = sorted({int(p) for b in range(B) for p in table[b] if p >= 0})
    assert torch.equal(got[0][0], got[1][0][:6 * B]) and torch.equal(got[0][1], got[1][1][:6 * B])
    for x in got[0][2]:
        assert torch.equal(got[0][2][x].view(torch.uint8)[pages], got[1][2][x].view(torch.uint8)[pages]), x
    tok, page = s["tok"].numpy(), s["page"].numpy()
    ang = np.concatenate([tok[:, None].astype(np.float64) * np.array([10000.0 ** (-j / 63) for j in range(63)]), (page % 2)[:, None]], axis=1)
    c, sn = np.cos(ang), np.sin(ang)
    for src, out, cc, ss in ((s["q"], got[1][0], c[:, None], sn[:, None]), (s["idx_q"], got[1][1], c, sn)):
        x = src.double().numpy()
        a, b = x[..., :64], x[..., 64:]
        w = np.concatenate([a * cc - b * ss, b * cc + a * ss], axis=-1)
        want, gap = bf16_rounded(w)
        # the reference's angles and products are themselves off by a few 2^-53 of 120000 rad and of the terms
        sure = gap > 2.0 ** -34 * np.concatenate([np.abs(a) + np.abs(b)] * 2, axis=-1)
        assert sure.mean() > 0.9999
        assert (out.double().cpu().numpy() == want)[sure].all()


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 3.3e38, -3.3e38, 0.0, 1e-38, -3e-40, 1e-30])
def test_append_extreme_values_alike_in_both_kernels(uocr, cuda_device, value):
    """Infinities, NaN, the largest and the smallest numbers in either half of q, idx_q, k, idx_k and v, at position 0 too (a sine
    of 0): the kernel for few tokens and the one for many give the same, NaN where the other has NaN."""
    H, B = 2, 12
    lens, new = [6 + 3 * b for b in range(B)] + [60], [6] * B + [60]
    s, table, starts, n = append_state(81, H, lens, new)
    s["tok"][::4] = 0
    s["page"][::3] = 0
    for name in ("q", "k_new", "v_new", "idx_q", "idx_k_new"):
        x = s[name].view(n, -1, 128)
        x[1::6, :, 3] = value              # first half, second half, both, whole rows
        x[2::6, :, 67] = value
        x[3::6, :, 5], x[3::6, :, 69] = value, -value
        x[4::6] = value
        x[::4, :, 63], x[1::4, :, 127] = value, value      # the page's pair
    few = {x: (v[:6 * B] if v.shape[0] == n else v) for x, v in s.items()}
    a = run_append(uocr, cuda_device, few, table[:B], lens[:B], starts[:B + 1])
    b = run_append(uocr, cuda_device, s, table, lens, starts)
    pages = sorted({int(p) for x in range(B) for p in table[x] if p >= 0})

    def alike(x, y):
        x, y = x.float(), y.float()
        return bool(((x == y) | (torch.isnan(x) & torch.isnan(y))).all())

    assert alike(a[0], b[0][:6 * B]) and alike(a[1], b[1][:6 * B])
    for x in a[2]:
        assert alike(a[2][x][pages], b[2][x][pages]), x
    if not math.isfinite(value):
        assert torch.isinf(a[0].float()).any() == math.isinf(value)


def test_append_extreme_values(uocr, cuda_device):
    lens, H = [40, 64], 2
    s, table, starts, n = append_state(6, H, lens, [20, 64])
    s["k_new"][3] = 0
    s["v_new"][:20] = 0                       # an older page, all new rows zero
    s["v_new"][20:52, 1] = 0                  # a fresh page of zeros: the least scale
    s["v_new"][60, 0, 5] = math.nan
    s["v_new"][61, 0, 6] = math.inf
    s["v_new"][62, 0, 7] = -math.inf
    s["v_new"][63, 1] = 1e38
    s["k_new"][70, 0] = 3e38
    s["k_new"][71, 1] = 1e-40
    s["k_scale"][int(table[0, 0])] = 0.013    # not a power of two
    want = ref.append(s, starts, lens, table)
    got = run_append(uocr, cuda_device, s, table, lens, starts)
    check_append(s, got, want, (torch.full_like(s["q"], 7.0), torch.full_like(s["idx_q"], 7.0)))


def test_append_codes_alike_in_both_kernels_over_many_values(uocr, cuda_device):
    """30 million keys as 6 a sequence (the kernel for few) and beside a longer sequence (the one for many): a sum that
    is off by 2^-25 of its terms would give another code for some ten of them."""
    H, B, dev = 16, 2500, cuda_device
    g = torch.Generator(device=dev).manual_seed(82)
    n = 6 * B + 40
    rnd = lambda *shape: torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    q, k, v, iq, ik = rnd(n, H, 128), rnd(n, H, 128), rnd(n, H, 128), rnd(n, 128), rnd(n, 128)
    tok = torch.randint(0, 100000, (n,), generator=g, device=dev, dtype=torch.int32)
    table = torch.arange(2 * (B + 1), device=dev, dtype=torch.int32).reshape(B + 1, 2)
    lens = torch.tensor([6] * B + [40], device=dev, dtype=torch.int32)
    starts = torch.tensor([6 * b for b in range(B + 1)] + [n], device=dev, dtype=torch.int32)
    P, got = 2 * (B + 1), []
    for b in (B, B + 1):
        m = int(starts[b])
        c = [torch.zeros((P, H, 32, 128), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
        s = [torch.zeros((P, H), device=dev) for _ in range(2)]
        cik = torch.zeros((P, 32, 128), dtype=torch.bfloat16, device=dev)
        uocr.rope_append_kv8(q[:m], iq[:m], k[:m], v[:m], ik[:m], tok[:m], tok[:m], table[:b], lens[:b], *c, *s, cik, starts[:b + 1],
                             q_out=torch.empty_like(q[:m]), idx_q_out=torch.empty_like(iq[:m]))
        got.append([x.view(torch.uint8)[:2 * B] for x in (*c, *s)])
    assert int((got[0][0] & 0x7F).max()) > 100
    for a, b in zip(*got):
        assert torch.equal(a, b), int((a != b).sum())


@pytest.mark.parametrize("old", [-0.25, -0.013, -3.0, -1e30, -1e-40, 0.0, 1e-40, 3e38, -3e38])
@pytest.mark.parametrize("n", [1, 20])       # the kernel for few tokens; the one for many
def test_append_to_a_page_of_any_finite_scale(uocr, cuda_device, old, n):
    """Older rows keep their values (to e4m3's rounding under the new scale), also under a negative scale, which their
    new codes' signs take up."""
    H, lens = 3, [11 + n]
    s, table, starts, _ = append_state(83, H, lens, [n])
    page = int(table[0, 0])
    s["k_scale"][page], s["v_scale"][page] = old, old
    old = float(s["k_scale"][page, 0])
    _, _, got = run_append(uocr, cuda_device, s, table, lens, starts)
    rot = [ref.rotate(s["k_new"][i].double(), int(s["tok"][i]), int(s["page"][i])) for i in range(n)]
    for x, rows in (("k", np.stack(rot)), ("v", s["v_new"].double().numpy())):
        for h in range(H):
            scale = max(ref.need_scale(rows[:, h]), min(ref.pow2_at_least(abs(old)), 2.0 ** 127))
            assert float(got[x + "_scale"][page, h]) == scale
            before = ref.GRID[s[x].view(torch.uint8).numpy()[page, h, :11]] * old
            codes = got[x].view(torch.uint8)[page, h].numpy()
            assert (ref.GRID[codes[:11]] == ref.GRID[ref.encode(before / scale)]).all()
            assert (ref.GRID[codes[11:11 + n]] == ref.GRID[ref.encode(rows[:, h] / scale)]).all()


@pytest.mark.parametrize("n", [1, 20])       # the kernel for few tokens; the one for many
def test_append_rescales_older_codes_with_one_rounding(uocr, cuda_device, n):
    """Scales that take a code within 2^-24 of a midpoint of e4m3, on either side: 28 bits that round to the midpoint
    itself in fp32."""
    scales = [np.float32((k + 0.5) / c * 2.0 ** -j) for c in range(9, 16) for k in range(8, 16) for j in (3, 4)]
    H, lens = len(scales) // 7, [11 + n]
    for part in range(7):
        s, table, starts, _ = append_state(84 + part, H, lens, [n])
        page = int(table[0, 0])
        for x in "kv":
            s[x + "_scale"][page] = torch.tensor(scales[part * H:(part + 1) * H])
            s[x][page, :, :11] = torch.arange(8, 16).repeat(16).float().to(ref.E4M3)      # 8 .. 15, exactly
            s[x + "_new"] *= 2.0 ** -20                                                   # they do not raise the scale
        _, _, got = run_append(uocr, cuda_device, s, table, lens, starts)
        beside = 0
        for x in "kv":
            for h in range(H):
                old, scale = float(s[x + "_scale"][page, h]), float(got[x + "_scale"][page, h])
                assert scale == ref.pow2_at_least(old)
                before = ref.GRID[s[x].view(torch.uint8).numpy()[page, h, :11]] * old / scale
                codes = got[x].view(torch.uint8)[page, h, :11].numpy()
                assert (ref.GRID[codes] == ref.GRID[ref.encode(before)]).all()
                beside += int((ref.encode(before) != ref.encode(before.astype(np.float32))).sum())
        assert beside > 0


def test_append_to_a_padded_batch(uocr, cuda_device):
    """One token a sequence, some places of the batch empty: nothing of theirs is touched and nothing flagged; a length
    below 0 still is."""
    lens, H = [33, 0, 1, 0, 64], 3
    s, table, starts, n = append_state(92, H, lens, [1] * 5)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = run_append(uocr, cuda_device, s, table, lens, None, dev_err=err, null_start=True)
    assert int(err) == 0
    want = ref.append(s, starts, lens, table)
    check_append(s, got, want, (torch.full_like(s["q"], 7.0), torch.full_like(s["idx_q"], 7.0)))
    assert (got[0][[1, 3]] == 7).all() and (got[1][[1, 3]] == 7).all()
    lens[3] = -1
    run_append(uocr, cuda_device, s, table, lens, None, dev_err=err, null_start=True)
    assert int(err) == uocr.DEVERR_POS


def test_append_bad_sequences_are_skipped(uocr, cuda_device):
    lens = [40, 5, 96, 70]
    s, table, starts, n = append_state(7, 2, lens, [10, 5, 40, 3])
    lens[1] = 4                                  # more new tokens than the sequence has
    table[2, 2] = 10 ** 7                        # a page outside the pool: its q rows are still rotated
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    want = ref.append(s, starts, lens, table)
    got = run_append(uocr, cuda_device, s, table, lens, starts, dev_err=err)
    assert int(err) == uocr.DEVERR_POS | uocr.DEVERR_PAGE
    check_append(s, got, want, (torch.full_like(s["q"], 7.0), torch.full_like(s["idx_q"], 7.0)))


@pytest.mark.parametrize("starts", [[0, 12, 5, 20], [-4, 3, 9, 20], [0, 8, 16, 999], [9, 9, 9, 9]])
def test_append_starts_out_of_order_stay_in_bounds(uocr, cuda_device, starts):
    """Starts that do not ascend from 0 to n: what is not a sequence's own rows is skipped and flagged."""
    lens = [40, 50, 60]
    s, table, _, n = append_state(8, 1, lens, [7, 7, 6])
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    run_append(uocr, cuda_device, s, table, lens, starts, dev_err=err)
    assert int(err) == (0 if starts == [9, 9, 9, 9] else uocr.DEVERR_POS)


# ---------------------------------------------------------------------------------------- eviction
def run_evict(uocr, dev, mass, table, lens, keep, sink, in_place=False):
    m, t, n = to(dev, mass, table, lens)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kw = dict(new_mass=m, new_table=t, new_lens=n) if in_place else {}
    r = uocr.evict_blocks(m, t, n, keep, n_sink=sink, dev_err=err, **kw)
    return [x.cpu() for x in r], int(err)


@pytest.mark.parametrize("mb,H", [(1, 1), (9, 3), (33, 10), (1024, 2), (1025, 5), (5000, 3)])
@pytest.mark.parametrize("kind", ["long_tail", "ties", "zeros", "odd_values"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(uocr, cuda_device, mb, H, kind, in_place):
    g = torch.Generator().manual_seed(mb * 7 + H)
    B = 5
    mass = torch.exp(2 * torch.randn((B, H, mb), generator=g))
    if kind == "ties":
        mass = torch.randint(0, 3, (B, H, mb), generator=g).float()
    elif kind == "zeros":
        mass[torch.rand((B, 1, mb), generator=g).expand(B, H, mb) < 0.9] = 0.0
    elif kind == "odd_values":
        mass[torch.rand(mass.shape, generator=g) < 0.1] *= -1
        mass[torch.rand(mass.shape, generator=g) < 0.02] = math.nan
        mass[:, 0][torch.rand((B, mb), generator=g) < 0.02] = math.inf
        mass[torch.rand(mass.shape, generator=g) < 0.1] = -0.0
    table = torch.randint(0, 1 << 20, (B, mb), generator=g, dtype=torch.int32)
    lens = torch.tensor([mb * BLOCK, 0, max(1, mb * BLOCK - 17), mb * BLOCK // 2 + 1, 1], dtype=torch.int32)
    for keep, sink in ((4, 0), (5, 1), (max(6, mb // 3), 2), (mb + 4, 0)):
        if sink > mb:
            continue
        want = ref.evict(mass, table, lens, keep, sink)
        got, err = run_evict(uocr, cuda_device, mass, table, lens, keep, sink, in_place)
        assert err == 0
        for w, x, name in zip(want, got, ("mass", "table", "lens", "freed", "n_freed")):
            assert torch.equal(w.view(torch.int32) if w.is_floating_point() else w, x.view(torch.int32) if x.is_floating_point() else x), (name, keep, sink)


@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_tables_beyond_shared_memory(uocr, cuda_device, H, in_place):
    """Long tables take another launch plan; sequences that keep, cut a little and cut nearly everything."""
    g = torch.Generator().manual_seed(50 + H)
    B, mb = 3, 30001
    mass = torch.exp(2 * torch.randn((B, H, mb), generator=g))
    mass[:, :, ::3] = 0.0
    table = torch.randint(0, 1 << 20, (B, mb), generator=g, dtype=torch.int32)
    lens = torch.tensor([mb * BLOCK - 5, 9000 * BLOCK, 20000 * BLOCK + 1], dtype=torch.int32)
    for keep, sink in ((9500, 3), (29000, 0), (4, 0)):
        want = ref.evict(mass, table, lens, keep, sink)
        got, err = run_evict(uocr, cuda_device, mass, table, lens, keep, sink, in_place)
        assert err == 0
        for w, x, name in zip(want, got, ("mass", "table", "lens", "freed", "n_freed")):
            assert torch.equal(w, x), (name, keep, sink)


@pytest.mark.parametrize("mb,H", [(12000, 10), (16003, 4), (700, 64)])
def test_evict_on_the_largest_clusters(uocr, cuda_device, mb, H):
    """Tables of which only an eighth (a half, for many heads) fits in a CTA's shared memory."""
    g = torch.Generator().manual_seed(mb)
    mass = torch.exp(2 * torch.randn((2, H, mb), generator=g))
    mass[1] = torch.randint(0, 2, (H, mb), generator=g).float()
    table = torch.randint(0, 1 << 20, (2, mb), generator=g, dtype=torch.int32)
    lens = torch.tensor([mb * BLOCK - 40, mb * BLOCK], dtype=torch.int32)
    for keep, sink in ((mb // 4, 4), (mb - 3, 0)):
        want = ref.evict(mass, table, lens, keep, sink)
        got, err = run_evict(uocr, cuda_device, mass, table, lens, keep, sink, True)
        assert err == 0
        for w, x, name in zip(want, got, ("mass", "table", "lens", "freed", "n_freed")):
            assert torch.equal(w, x), (name, keep, sink)


def meet(calls, times):
    """Each call's arguments, times over from two threads of its own, all at once; the numbers of failed ones.  As the
    binding calls the library, without its checks, so that the threads meet."""
    import threading
    failed, ready = [], threading.Barrier(2 * len(calls))

    def work(call, args):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        args = args()
        ready.wait()
        failed.append(sum(call(*args, stream.cuda_stream) != 0 for _ in range(times)))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=x) for x in calls + calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return failed


def test_selection_from_several_threads(uocr, cuda_device):
    """Rows of very different widths (staged in 18 to 120 KiB of shared memory) by threads of their own: every call is
    launched and gives what it gives alone."""
    g = torch.Generator().manual_seed(61)
    calls, outs = [], []
    for mb in (4400, 30000, 17000):
        scores = torch.randn((3, mb), generator=g).to(cuda_device)
        lens = torch.tensor([mb * BLOCK, mb * BLOCK - 40, 5000], dtype=torch.int32, device=cuda_device)
        want = uocr.block_topk(scores, lens)

        def args(scores=scores, lens=lens, mb=mb, want=want):
            outs.append((torch.empty_like(want), want, scores, lens))
            return scores.data_ptr(), lens.data_ptr(), None, None, 3, 3, mb, outs[-1][0].data_ptr(), None

        calls.append((uocr.lib.uocr_block_topk, args))
    torch.cuda.synchronize()
    assert meet(calls, 3000) == [0] * 6
    assert len(outs) == 6 and all(torch.equal(a, b) for a, b, *_ in outs)


def test_evict_from_several_threads(uocr, cuda_device):
    """Tables of very different widths (shared memory from 9 to 190 KiB a CTA) evicted by threads of their own, each on
    its stream: every call is launched and gives what it gives alone."""
    import threading
    g = torch.Generator().manual_seed(60)
    jobs = []
    for mb, H in ((40, 1), (12000, 10), (700, 64), (40, 2)):
        mass = torch.exp(2 * torch.randn((2, H, mb), generator=g)).to(cuda_device)
        table = torch.randint(0, 1 << 20, (2, mb), generator=g, dtype=torch.int32).to(cuda_device)
        lens = torch.tensor([mb * BLOCK, mb * BLOCK - 40], dtype=torch.int32, device=cuda_device)
        want = [x.clone() for x in uocr.evict_blocks(mass, table, lens, mb // 2, n_sink=1)]
        jobs.append((mass, table, lens, mb // 2, want))
    torch.cuda.synchronize()
    wrong, ready = [], threading.Barrier(2 * len(jobs))

    def work(job):
        mass, table, lens, keep, want = job
        (B, H, mb), out = mass.shape, [torch.empty_like(x) for x in want]
        ws = torch.empty(uocr.evict_workspace_bytes(B, H, mb), dtype=torch.uint8, device=cuda_device)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        at = [x.data_ptr() for x in out]
        args = (mass.data_ptr(), table.data_ptr(), lens.data_ptr(), B, H, mb, keep, 1, *at, ws.data_ptr(), ws.numel(), None, stream.cuda_stream)
        call = uocr.lib.uocr_evict_blocks      # as the binding calls it, without its checks, so that the threads meet
        ready.wait()
        bad = sum(call(*args) != 0 for _ in range(3000))
        stream.synchronize()
        if bad or not all(torch.equal(a, b) for a, b in zip(want, out)):
            wrong.append((mb, H, bad))

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs + jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_evict_bad_lengths_copy_and_flag(uocr, cuda_device):
    mass, table = torch.rand((3, 2, 50)), torch.arange(150, dtype=torch.int32).reshape(3, 50)
    lens = torch.tensor([-1, 50 * BLOCK + 1, 1000], dtype=torch.int32)
    got, err = run_evict(uocr, cuda_device, mass, table, lens, 10, 0)
    assert err == uocr.DEVERR_POS
    for w, x in zip(ref.evict(mass, table, lens, 10, 0), got):
        assert torch.equal(w, x)


# --------------------------------------------------------------------- streams, graphs, used together
def test_binding_refusals(uocr, cuda_device):
    c = Case([300, 64], 2, seed=20)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    sel = c.select([299, 63]).to(cuda_device)
    mass = c.mass.to(cuda_device)
    seq = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    for bad in (dict(k_cache=k.view(torch.uint8)), dict(k_scale=ks[:-1].contiguous()), dict(k_scale=ks.double()), dict(v_cache=v[1:].contiguous()),
                dict(sel=sel[:, :15].contiguous()), dict(sel=sel.long()), dict(mass=mass[:, :, :-1].contiguous()), dict(mass=mass, q_seq=seq),
                dict(out=q[:1]), dict(q=q.transpose(0, 1)), dict(seq_lens=sl[:1]), dict(block_table=bt.long()), dict(q_pos=seq[:1]),
                dict(v_scale=vs.cpu()), dict(dev_err=torch.zeros(1, device=cuda_device)), dict(scale=math.nan)):
        a = dict(q=q, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_table=bt, seq_lens=sl, sel=sel)
        a.update(bad)
        with pytest.raises((ValueError, TypeError, uocr.UocrError)):
            uocr.sparse_attn_kv8(**a)
    with pytest.raises(uocr.UocrError):
        uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, ref_blocks=-1)
    with pytest.raises(uocr.UocrError):
        uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(uocr.UocrError):
        uocr.evict_blocks(mass, bt, sl, 3)
    with pytest.raises(uocr.UocrError):
        uocr.evict_blocks(mass, bt, sl, 8, new_table=bt, freed=bt)
    with pytest.raises(uocr.UocrError):
        uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, 2, seq, sel)
    assert uocr.sparse_attn_seq_kv8(q[:0], k, v, ks, vs, bt, sl, 0, seq[:0], sel[:0]).shape == (0, 2, 128)


def test_integers_past_32_bits(uocr, cuda_device):
    """Numbers of blocks past 32 bits mean what they say; a sequence or a sink past them is refused."""
    c = Case([900, 700], 2, seed=23)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    full = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl)
    for big in (1 << 31, 1 << 32, (1 << 32) + 1, (1 << 63) - 1):
        assert torch.equal(full, uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, ref_blocks=big))
        mass = c.mass.to(cuda_device)
        got = uocr.evict_blocks(mass, bt, sl, big, n_sink=1)
        assert torch.equal(got[0], mass) and torch.equal(got[1], bt) and torch.equal(got[2], sl) and (got[3] == -1).all() and (got[4] == 0).all()
    pos, sel = (sl[:1] - 1).expand(2).contiguous(), c.select([899, 899]).to(cuda_device)
    idx, idx_k = torch.zeros((2, 128), dtype=torch.bfloat16, device=cuda_device), torch.zeros((k.shape[0], 32, 128), dtype=torch.bfloat16, device=cuda_device)
    for bad in (1 << 31, 1 << 32, (1 << 32) + 1, -(1 << 32)):
        with pytest.raises(ValueError):
            uocr.sparse_attn_seq_kv8(q, k, v, ks, vs, bt, sl, bad, pos, sel)
        with pytest.raises(ValueError):
            uocr.sparse_prefill_kv8(q, k, v, ks, vs, idx, idx_k, bt, sl, bad, pos)
        with pytest.raises(ValueError):
            uocr.evict_blocks(c.mass.to(cuda_device), bt, sl, 8, n_sink=bad)
    for call in (lambda: uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, ref_blocks=-(1 << 32)), lambda: uocr.evict_blocks(c.mass.to(cuda_device), bt, sl, -(1 << 32) + 9)):
        with pytest.raises(ValueError):
            call()


def test_matches_the_bf16_cache_of_the_same_values(uocr, cuda_device):
    """Power-of-two scales make every cached value a bf16 number, so both caches hold the same keys and values."""
    c = Case([700, 1500, 90], 10, seed=21)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    kb = (k.float() * ks[:, :, None, None]).nan_to_num(0).to(torch.bfloat16)
    vb = (v.float() * vs[:, :, None, None]).nan_to_num(0).to(torch.bfloat16)
    g = torch.Generator().manual_seed(3)
    iq = torch.randn((3, 128), generator=g).to(torch.bfloat16).to(cuda_device)
    ik = torch.randn((k.shape[0], 32, 128), generator=g).to(torch.bfloat16).to(cuda_device)
    o8, s8 = uocr.sparse_decode_kv8(q, k, v, ks, vs, iq, ik, bt, sl)
    o16, s16 = uocr.sparse_decode(q, kb, vb, iq, ik, bt, sl)
    assert torch.equal(s8, s16)
    check_rows(c, o8, None, [(i, i, c.lens[i] - 1, s8[i].tolist()) for i in range(3)])
    assert (o8.float() - o16.float()).abs().max() <= 2.0 ** -7 * o16.float().abs().max()


def test_prefill_step_selects_like_the_bf16_one(uocr, cuda_device):
    n, total = 70, 2100
    c = Case([total], 3, seed=22, n_q=n)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    g = torch.Generator().manual_seed(4)
    iq = torch.randn((n, 128), generator=g).to(torch.bfloat16).to(cuda_device)
    ik = torch.randn((k.shape[0], 32, 128), generator=g).to(torch.bfloat16).to(cuda_device)
    pos = torch.arange(total - n, total, dtype=torch.int32, device=cuda_device)
    mass = c.mass.to(cuda_device)
    out, sel = uocr.sparse_prefill_kv8(q, k, v, ks, vs, iq, ik, bt, sl, 0, pos, mass=mass)
    zero = torch.zeros((k.shape[0], 3, 32, 128), dtype=torch.bfloat16, device=cuda_device)
    _, want = uocr.sparse_prefill(q, zero, zero, iq, ik, bt, sl, 0, pos)
    assert torch.equal(sel, want)
    sel = sel.cpu()
    check_rows(c, out, mass, [(i, 0, total - n + i, sel[i].tolist()) for i in range(n)], many=True)


def test_captured_replayed_and_on_another_stream(uocr, cuda_device):
    """A decode step (append, attention with totals, eviction) captured once and replayed on new contents, beside a
    second graph that shares the first one's workspace."""
    lens, H = [500, 1000], 3
    s, table, starts, n = append_state(30, H, lens, [1, 1])
    d = {k: v.to(cuda_device) for k, v in s.items()}
    bt, sl = table.to(cuda_device), torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    mb = table.shape[1]
    mass = torch.zeros((2, H, mb), device=cuda_device)
    ws = torch.empty(uocr.dense_kv8_workspace_bytes(2, H, mb), dtype=torch.uint8, device=cuda_device)
    ews = torch.empty(uocr.evict_workspace_bytes(2, H, mb), dtype=torch.uint8, device=cuda_device)
    qo, io = torch.empty_like(d["q"]), torch.empty_like(d["idx_q"])
    out, ev = torch.empty_like(d["q"]), [torch.empty_like(mass), torch.empty_like(bt), torch.empty_like(sl), torch.empty_like(bt), torch.empty_like(sl)]

    def step():
        uocr.rope_append_kv8(d["q"], d["idx_q"], d["k_new"], d["v_new"], d["idx_k_new"], d["tok"], d["page"], bt, sl, d["k"], d["v"],
                             d["k_scale"], d["v_scale"], d["idx_k"], q_out=qo, idx_q_out=io)
        uocr.dense_decode_kv8(qo, d["k"], d["v"], d["k_scale"], d["v_scale"], bt, sl, out=out, mass=mass, workspace=ws)
        uocr.evict_blocks(mass, bt, sl, 12, n_sink=1, new_mass=ev[0], new_table=ev[1], new_lens=ev[2], freed=ev[3], n_freed=ev[4], workspace=ews)

    start = {k: v.clone() for k, v in d.items()}

    def reset():
        for k, v in start.items():
            d[k].copy_(v)
        mass.zero_()

    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (out, mass, *ev)]
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for a, b in zip(want, (out, mass, *ev)):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        reset()
        for x in (out, *ev):
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (out, mass, *ev)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [20, 150])     # a query at a time; block by block
def test_prefill_and_decode_captured_and_replayed_on_new_contents(uocr, cuda_device, n):
    """Two graphs on one workspace, replayed in turn after the queries, caches and lengths have changed."""
    H, total = 10, 3000
    c, other = Case([total, 777], H, seed=61, n_q=n), Case([total - 200, 900], H, seed=62, n_q=n, max_blocks=94)
    assert c.mb == other.mb and c.k.shape[0] >= other.k.shape[0]
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    g = torch.Generator().manual_seed(63)
    iq, ik = (torch.randn(s, generator=g).to(torch.bfloat16).to(cuda_device) for s in ((n, 128), (k.shape[0], 32, 128)))
    pos = torch.arange(total - n - 200, total - 200, dtype=torch.int32, device=cuda_device)
    mass = torch.zeros((2, H, c.mb), device=cuda_device)
    ws = torch.empty(uocr.prefill_kv8_workspace_bytes(n, H, c.mb), dtype=torch.uint8, device=cuda_device)
    out, sel = torch.empty_like(q), torch.empty((n, 16), dtype=torch.int32, device=cuda_device)
    dout, dsel = torch.empty_like(q[:2]), torch.empty_like(sel[:2])
    dws = torch.empty(uocr.workspace_bytes(2, H, c.mb), dtype=torch.uint8, device=cuda_device)

    def step():
        uocr.sparse_prefill_kv8(q, k, v, ks, vs, iq, ik, bt, sl, 0, pos, out=out, sel=sel, mass=mass, workspace=ws)
        uocr.sparse_decode_kv8(q[:2], k, v, ks, vs, iq[:2], ik, bt, sl, out=dout, sel=dsel, mass=mass, workspace=dws)

    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step()
    for case in (c, other, c):
        pages = case.k.shape[0]
        for have, want in ((q, case.q), (k[:pages], case.k), (v[:pages], case.v), (ks[:pages], case.ks), (vs[:pages], case.vs), (bt, case.table),
                           (sl, case.sl)):
            have.copy_(want)
        mass.zero_()
        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in (out, sel, dout, dsel, mass)]
        for graph in graphs:
            mass.zero_()
            for x in (out, sel, dout, dsel):
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(want, (out, sel, dout, dsel, mass)):
                assert torch.equal(a, b)
    base = total - n - 200
    rows = [(i, 0, base + i, want[1][i].tolist()) for i in range(n)]
    case = Case([total, 777], H, seed=61, n_q=n)
    check_rows(case, want[0], None, rows, many=True)
    assert abs(float(mass[0].sum()) - H * (n + 1)) < 1e-3 * H * (n + 1)


def test_memory_of_a_call_on_another_stream_is_not_given_out(uocr, cuda_device, monkeypatch):
    """A call on a given stream that allocates for itself: the workspace that it drops and outputs that the caller
    drops stay taken until that stream has run it."""
    c = Case([2000], 10, seed=35)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    spaces = []
    real = uocr._space

    def spy(*args):
        t = real(*args)
        spaces.append((t.data_ptr(), t.numel()))
        return t

    monkeypatch.setattr(uocr, "_space", spy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    out = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, stream=side)
    at, size = spaces[0]
    dropped = out.data_ptr()
    del out
    again = torch.empty(size, dtype=torch.uint8, device=cuda_device)
    other = torch.empty_like(q)
    busy = not side.query()
    side.synchronize()
    assert busy, "the stream was done before the allocations"
    assert again.data_ptr() != at and other.data_ptr() != dropped


def test_a_call_on_another_stream_takes_no_memory_with_work_queued_on_the_current_one(uocr, cuda_device):
    """Tensors dropped while the current stream still has to read them: a call on another stream that allocates the same
    sizes writes elsewhere.  And the other way round: an output dropped while the current stream still reads it."""
    c = Case([2000], 10, seed=36)
    q, k, v, ks, vs, bt, sl = c.gpu(cuda_device)
    mass = c.mass.to(cuda_device)
    g = torch.Generator().manual_seed(1)
    iq, ik = (torch.randn(s, generator=g).to(torch.bfloat16).to(cuda_device) for s in ((1, 128), (k.shape[0], 32, 128)))
    n = 100
    qn, pos = q.expand(n, -1, -1).contiguous(), torch.arange(1900, 2000, dtype=torch.int32, device=cuda_device)
    sel = c.select([1999] * n)
    sel = torch.where(sel > pos.cpu()[:, None] // BLOCK, -1, sel).to(cuda_device)
    iqn = iq.expand(n, -1).contiguous()
    calls = {
        "sparse": (lambda s: (uocr.sparse_attn_kv8(q, k, v, ks, vs, bt, sl, sel[:1], stream=s),), 0),
        "decode": (lambda s: uocr.sparse_decode_kv8(q, k, v, ks, vs, iq, ik, bt, sl, stream=s), uocr.workspace_bytes(1, 10, c.mb)),
        "dense": (lambda s: (uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, stream=s),), uocr.dense_kv8_workspace_bytes(1, 10, c.mb)),
        "seq": (lambda s: (uocr.sparse_attn_seq_kv8(qn, k, v, ks, vs, bt, sl, 0, pos, sel, stream=s),), uocr.sparse_attn_seq_kv8_workspace_bytes(n, 10, c.mb)),
        "prefill": (lambda s: uocr.sparse_prefill_kv8(qn, k, v, ks, vs, iqn, ik, bt, sl, 0, pos, stream=s), uocr.prefill_kv8_workspace_bytes(n, 10, c.mb)),
        "evict": (lambda s: uocr.evict_blocks(mass, bt, sl, 20, stream=s), uocr.evict_workspace_bytes(1, 10, c.mb)),
    }
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, (call, space) in calls.items():
        want = [x.clone() for x in call(None)]
        torch.cuda.synchronize()
        sizes = [x.numel() * x.element_size() for x in want] + [space] * (space > 0)
        torch.cuda.empty_cache()
        temps = [torch.full((x,), 0x5A, dtype=torch.uint8, device=cuda_device) for x in sizes]
        keep = [torch.zeros_like(t) for t in temps]
        torch.cuda.synchronize()
        torch.cuda._sleep(80_000_000)
        for a, b in zip(keep, temps):
            a.copy_(b)
        del temps, a, b
        got = call(side)
        side.synchronize()
        busy = not torch.cuda.current_stream().query()
        assert busy, "the current stream was done before the call on the other"
        torch.cuda.synchronize()
        assert all((x == 0x5A).all() for x in keep), name
        assert all(torch.equal(x, y) for x, y in zip(got, want)), name
        torch.cuda._sleep(20_000_000)
        later = [x.clone() for x in got]
        del got
        other = call(side)          # must not be given the memory that the clones still have to read
        for x in other:
            with torch.cuda.stream(side):
                x.zero_()
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(later, want)), name


def test_prompt_decode_evict_decode(uocr, cuda_device):
    """The operators as a server uses them: a prompt appended and attended in two chunks, decode steps, an eviction in
    place, pages freed, more decode steps on the shorter table; every attention against the 64-bit form on the cache
    as it stands, every total and every table against the plain ones."""
    dev, H, keep, sink = cuda_device, 4, 14, 1
    g = torch.Generator().manual_seed(40)
    mb, pages = 40, 60
    rnd = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16)  # noqa: E731
    c = Case([0, 0], H, seed=41, max_blocks=mb)      # holder of the caches on the CPU side
    c.k = torch.full((pages, H, 32, 128), math.nan).to(torch.float8_e4m3fn)
    c.v, c.ks, c.vs = c.k.clone(), torch.full((pages, H), math.nan), torch.full((pages, H), math.nan)
    k, v, ks, vs = to(dev, c.k, c.v, c.ks, c.vs)
    ik = torch.zeros((pages, 32, 128), dtype=torch.bfloat16, device=dev)
    free = torch.randperm(pages, generator=g).tolist()
    table = torch.full((2, mb), -1, dtype=torch.int32)
    lens, true_pos = [0, 0], [0, 0]
    mass = torch.zeros((2, H, mb), device=dev)
    c.mass = torch.zeros((2, H, mb))

    def grow(b, n):
        for j in range(-(-lens[b] // 32), -(-(lens[b] + n) // 32)):
            table[b, j] = free.pop()
        lens[b] += n

    def mirror():
        c.k, c.v, c.ks, c.vs = [x.cpu() for x in (k, v, ks, vs)]
        c.table = table

    def append(news):
        for b, n in enumerate(news):
            grow(b, n)
        n = sum(news)
        q, iq, kn, vn, ikn = rnd(n, H, 128), rnd(n, 128), rnd(n, H, 128), rnd(n, H, 128), rnd(n, 128)
        tok = torch.cat([torch.arange(true_pos[b], true_pos[b] + m, dtype=torch.int32) for b, m in enumerate(news)])
        for b, m in enumerate(news):
            true_pos[b] += m
        st = torch.tensor([0, news[0], n], dtype=torch.int32, device=dev)
        q, iq, kn, vn, ikn, tok = [x.to(dev) for x in (q, iq, kn, vn, ikn, tok)]
        bt, sl = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
        uocr.rope_append_kv8(q, iq, kn, vn, ikn, tok, torch.zeros_like(tok), bt, sl, k, v, ks, vs, ik, st)
        return q, iq, bt, sl

    for news in ([150, 33], [300, 77]):
        q, iq, bt, sl = append(news)
        mirror()
        c.q = q.cpu()
        at = 0
        for b, n in enumerate(news):
            pos = torch.arange(lens[b] - n, lens[b], dtype=torch.int32, device=dev)
            out, sel = uocr.sparse_prefill_kv8(q[at:at + n], k, v, ks, vs, iq[at:at + n], ik, bt, sl, b, pos, mass=mass)
            full = torch.zeros_like(c.q)
            full[at:at + n] = out.cpu()
            check_rows(c, full, mass, [(at + i, b, int(pos[i]), sel[i].tolist()) for i in range(n)], many=True)
            c.mass = mass.cpu()
            at += n

    def decode(steps):
        for x in range(steps):
            q, iq, bt, sl = append([1, 1])
            mirror()
            c.q = q.cpu()
            if x % 2:
                out = uocr.dense_decode_kv8(q, k, v, ks, vs, bt, sl, mass=mass)
                rows = [(b, b, lens[b] - 1, list(range(-(-lens[b] // 32)))) for b in range(2)]
            else:
                out, sel = uocr.sparse_decode_kv8(q, k, v, ks, vs, iq, ik, bt, sl, mass=mass)
                rows = [(b, b, lens[b] - 1, sel[b].tolist()) for b in range(2)]
            check_rows(c, out, mass, rows)
            c.mass = mass.cpu()

    decode(5)
    bt, sl = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    want = ref.evict(mass.cpu(), table, torch.tensor(lens, dtype=torch.int32), keep, sink)
    got = uocr.evict_blocks(mass, bt, sl, keep, n_sink=sink, new_mass=mass, new_table=bt, new_lens=sl)
    for a, b in zip(want, got):
        assert torch.equal(a, b.cpu())
    assert got[4].tolist() == [1, 0] or got[4][0] > 0
    for b in range(2):
        free += [int(x) for x in got[3][b, :int(got[4][b])]]
    table.copy_(bt.cpu())
    lens[:] = sl.tolist()
    c.mass = mass.cpu()
    assert -(-lens[0] // 32) == keep
    decode(4)
