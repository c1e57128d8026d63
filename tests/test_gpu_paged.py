"""The paged 4-bit memory on the GPU against the oracle: page tables and slot maps, quantised
rows bit by bit, selections exactly, attention in fp64.

Tolerance of attention, in units of 2^-24 of U, the largest sum of |products| behind a logit
(PagedModel.attend): q is held as two 11-bit halves (4 units), each group's two matrix products
and their sum are rounded or cut at 2^-23 (2 x 2 + 2 units a group, at most 4 groups folded by
sums that each add one: bounded by 12 in all since the groups' parts add up to U), the factor
(scale * log2 e * 2^n) and its product 4: at most 24.  An error x of a logit moves a weight by the
factor e^x, so an output by at most 2 x of the largest |v|; the weights' halves, exp2 and the
normalisation add 8 units of 2^-22, and each strip summed one more of 2^-23 (cut accumulators)."""
import math

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu


def bf16(x):
    return O.round_bf16(x)


def cuda(x, dtype="f32"):
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    return t.bfloat16() if dtype == "bf16" else t


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(r, shape, dtype="f32"):
    x = r.normal(size=shape).astype(np.float32)
    return bf16(x) if dtype == "bf16" else x


class Pair:
    """A store and its model, driven by the same calls."""

    def __init__(self, rba, seed, *, heads=2, group=2, dim=128, page=16, n_pages=64, requests=3,
                 columns=24, dtype="bf16"):
        self.r = np.random.default_rng(seed)
        self.dtype, self.heads, self.group, self.dim, self.page = dtype, heads, group, dim, page
        self.m = O.PagedModel(heads, dim, page, n_pages, requests, columns)
        self.st = rba.PagedStore(n_q_heads=heads * group, n_kv_heads=heads, head_dim=dim,
                                 page_size=page, n_pages=n_pages, max_requests=requests,
                                 max_pages=columns, dtype=dtype)

    def grow(self, new, pad=3, k=None, v=None):
        total = sum(new)
        slots, starts = self.st.extend(i32(new), total + pad)
        want = self.m.extend(new, total + pad)
        assert slots.tolist() == want + [-1] * pad
        assert starts.tolist() == [0] + np.cumsum(new).tolist()
        k = rows(self.r, (total + pad, self.heads, self.dim), self.dtype) if k is None else k
        v = rows(self.r, (total + pad, self.heads, self.dim), self.dtype) if v is None else v
        self.st.append(slots, cuda(k, self.dtype), cuda(v, self.dtype))
        self.m.append(want, k, v)
        self.same_tables()
        return slots

    def same_tables(self):
        assert self.st.lens.tolist() == self.m.lens
        n = int(self.st.n_free)
        assert self.st.free[:n].tolist() == self.m.free
        for r, t in enumerate(self.m.tables):
            assert self.st.table[r, :len(t)].tolist() == t

    def queries(self, scale=1.0):
        q = rows(self.r, (len(self.m.lens), self.heads * self.group, self.dim), self.dtype) * \
            np.float32(scale)
        return q, cuda(q, self.dtype)

    def same_attention(self, q, qd, idx, sink, window, scale=None, **kw):
        scale = self.dim ** -0.5 if scale is None else scale
        out, lse = self.st.attend(qd, None if idx is None else i32(idx), sink, window, scale=scale,
                                  **kw)
        self.st.check()
        ref, rl, vmax, unit = self.m.attend(q, idx, sink, window, scale)
        strips = max(self.m.lens) / 16 + 1
        dx = 24 * unit * 2.0 ** -24
        tol = vmax * (2 * dx + 8 * 2.0 ** -22 + strips * 2.0 ** -23)
        err = np.abs(out.cpu().numpy() - ref).max()
        assert err <= tol, (err, tol)
        seen = np.isfinite(rl)
        got = lse.cpu().numpy()
        assert np.array_equal(np.isneginf(got), ~seen)
        top = np.abs(rl[seen]).max() if seen.any() else 0
        assert np.abs(got[seen] - rl[seen]).max(initial=0) <= dx + (top + 4) * 2.0 ** -22
        return out, lse


# ---------------------------------------------------------------------------------------------
# tables

@pytest.mark.parametrize("requests,page,biggest", [(1, 1, 5), (3, 7, 40), (40, 16, 300),
                                                   (1025, 3, 9), (4096, 2, 3)])
def test_tables_follow_the_model(rba, requests, page, biggest):
    r = np.random.default_rng(requests)
    n_pages = requests * (-(-4 * biggest // page))
    m = O.PagedModel(1, 4, page, n_pages, requests, -(-4 * biggest // page))
    st = rba.PagedStore(n_q_heads=1, n_kv_heads=1, head_dim=4, page_size=page, n_pages=n_pages,
                        max_requests=requests, max_pages=m.columns)
    for step in range(8):
        if step % 3 == 2:
            keep = [int(r.integers(0, n + 2)) for n in m.lens]
            st.truncate(i32(keep))
            m.truncate(keep)
        else:
            new = r.integers(0, biggest + 1, requests) * (r.random(requests) < 0.7)
            new = [int(min(x, m.columns * page - n)) for x, n in zip(new, m.lens)]
            slots, starts = st.extend(i32(new), sum(new) + step)
            want = m.extend(new, sum(new) + step)
            assert want is not None
            assert slots.tolist() == want + [-1] * step
            assert starts.tolist() == np.concatenate([[0], np.cumsum(new)]).tolist()
        st.check()
        assert st.lens.tolist() == m.lens
        n = int(st.n_free)
        assert n == len(m.free) and st.free[:n].tolist() == m.free
        table = st.table.cpu().numpy()
        for i, t in enumerate(m.tables):
            assert table[i, :len(t)].tolist() == t


def test_tables_of_fewer_requests_leave_the_others(rba):
    p = Pair(rba, 1, requests=4)
    p.grow([5, 20, 3, 30])
    slots, _ = p.st.extend(i32([1, 12]), 13)
    p.m.tables, rest = p.m.tables[:2], p.m.tables[2:]
    want = p.m.extend([1, 12], 13)
    p.m.tables += rest
    assert slots.tolist() == want
    p.same_tables()
    p.st.truncate(i32([2]))
    assert p.st.lens.tolist() == [2, 32, 3, 30]


@pytest.mark.parametrize("new,n_slots", [([40, 0, 0], 50), ([9, 9, 9], 26), ([-1, 2, 0], 9),
                                         ([2 ** 31 - 1, 2 ** 31 - 1, 5], 9), ([13, 12, 1], 30)])
def test_refused_extension_changes_nothing(rba, new, n_slots):
    # 6 pages of 8 and 4 columns: too long a request, too few slots, a negative and an enormous
    # count, more pages than are free
    st = rba.PagedStore(n_q_heads=1, n_kv_heads=1, head_dim=64, page_size=8, n_pages=6,
                        max_requests=3, max_pages=4)
    st.extend(i32([8, 9, 0]), 17)
    before = [t.clone() for t in (st.lens, st.n_free, st.free, st.table)]
    slots, starts = st.extend(i32(new), n_slots)
    assert slots.tolist() == [-1] * n_slots and starts.tolist() == [0] * 4
    assert all(torch.equal(a, b) for a, b in zip(before, (st.lens, st.n_free, st.free, st.table)))
    with pytest.raises(rba.RbaError) as e:
        st.check()
    assert e.value.status == rba.ERR_BOUNDS
    st.check()  # cleared


def test_refused_truncation_changes_nothing(rba):
    st = rba.PagedStore(n_q_heads=1, n_kv_heads=1, head_dim=64, page_size=8, n_pages=6,
                        max_requests=2, max_pages=4)
    st.extend(i32([8, 9]), 17)
    before = [t.clone() for t in (st.lens, st.n_free, st.free)]
    st.truncate(i32([0, -1]))
    assert all(torch.equal(a, b) for a, b in zip(before, (st.lens, st.n_free, st.free)))
    with pytest.raises(rba.RbaError):
        st.check()


# ---------------------------------------------------------------------------------------------
# rows

SHAPES = [(2, 128, 16, "bf16"), (1, 64, 16, "f32"), (3, 100, 50, "f32"), (2, 36, 7, "bf16"),
          (2, 96, 1, "bf16"), (1, 4, 24, "f32"), (5, 128, 33, "f32")]


@pytest.mark.parametrize("heads,dim,page,dtype", SHAPES)
def test_rows_are_stored_bit_by_bit(rba, heads, dim, page, dtype):
    p = Pair(rba, dim + page, heads=heads, dim=dim, page=page, dtype=dtype, n_pages=40,
             columns=40)
    kept = {}
    p.st.pool.fill_(0xA5)  # what no row covers stays as it was
    for new in ([3, 0, page], [1, page + 1, 0], [2 * page, 1, 1]):
        k, v = (rows(p.r, (sum(new) + 3, heads, dim), dtype) * np.float32(3) for _ in range(2))
        if dtype == "bf16":
            k, v = bf16(k), bf16(v)
        slots = p.grow(new, k=k, v=v).tolist()
        kept.update({s: (k[i], v[i]) for i, s in enumerate(slots) if s >= 0})
    p.st.check()
    pool = p.st.pool.cpu().numpy()
    P = p.st.pitch
    for page_no in range(40):
        for h in range(heads):
            for s in range(-(-page // 16)):
                own = [kept.get(page_no * page + s * 16 + t) if s * 16 + t < page else None
                       for t in range(16)]
                image, mask = O.strip_image(
                    *([None if x is None else O.quantise_row(x[w][h]) for x in own]
                      for w in (0, 1)), P)
                want = (image & mask) | (0xA5 & ~mask)
                assert np.array_equal(pool[page_no, h, s], want), (page_no, h, s)
    rep = p.st.rep.cpu().numpy()
    assert p.m.reps
    for page_no in range(40):
        if page_no in p.m.reps:
            # a mean of `page` stored values in 32 bits: page + 2 roundings of at most |value|
            top = np.abs([p.m.rows[page_no * page + i][0] for i in range(page)]).max()
            err = np.abs(rep[page_no, :, :dim] - p.m.reps[page_no]).max()
            assert err <= top * (page + 2) * 2.0 ** -24
            assert not rep[page_no, :, dim:].any()
        else:
            assert not rep[page_no].any()
    # read back, in any order, with repeats and none
    order = p.r.permutation(list(kept)).tolist()[:37]
    order = order + [-1] + order[:2]
    k, v = p.st.read(i32(order))
    for got, w in ((k, 0), (v, 1)):
        want = np.stack([p.m.rows[s][w] if s >= 0 else np.zeros((heads, dim)) for s in order])
        want = torch.from_numpy(want).float().to(got.dtype)  # (c s fits 32 bits: 4 + 8 bits)
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("heads,dim,page,dtype,n", [(64, 64, 16, "bf16", 40), (32, 100, 50, "f32", 90),
                                                    (24, 128, 7, "bf16", 131),
                                                    (40, 36, 33, "f32", 61),
                                                    (64, 128, 24, "bf16", 100),
                                                    (96, 64, 40, "f32", 160),
                                                    (160, 64, 128, "bf16", 260)])
@pytest.mark.parametrize("scattered", [True, False])
def test_rows_of_many_heads_are_stored_bit_by_bit(rba, heads, dim, page, dtype, n, scattered):
    """More (row, head) pairs than a CTA each, to sixteen slots a CTA: slots in no order, alone, in
    runs up and down, or all in a row, -1 between them."""
    r = np.random.default_rng(n)
    n_pages = -(-4 * n // page)
    st = rba.PagedStore(n_q_heads=heads, n_kv_heads=heads, head_dim=dim, page_size=page,
                        n_pages=n_pages, max_requests=1, max_pages=n_pages, dtype=dtype)
    free = r.permutation(n_pages * page // 4)[:n // 2] * 4  # one row of four each
    run = np.arange(n - n // 2) // 2 * 4 + 1 + np.arange(n - n // 2) % 2  # two rows beside them
    slots = np.concatenate([free, run[::-1][:len(run) // 3], run[:len(run) - len(run) // 3]])
    if not scattered:
        slots = np.arange(5, 5 + n)
    slots[5::11 if scattered else 57] = -1
    k, v = (rows(r, (n, heads, dim), dtype) for _ in range(2))
    if dtype == "bf16":
        k, v = bf16(k), bf16(v)
    st.pool.fill_(0xA5)
    st.append(i32(slots), cuda(k, dtype), cuda(v, dtype))
    st.check()
    kept = {int(s): i for i, s in enumerate(slots) if s >= 0}
    assert len(kept) == (slots >= 0).sum()
    pool = st.pool.cpu().numpy()
    for page_no in range(n_pages):
        for s in range(-(-page // 16)):
            own = [kept.get(page_no * page + s * 16 + t) if s * 16 + t < page else None
                   for t in range(16)]
            if all(i is None for i in own):
                assert (pool[page_no, :, s] == 0xA5).all()
                continue
            for h in r.permutation(heads)[:6]:
                image, mask = O.strip_image(
                    *([None if i is None else O.quantise_row(x[i, h]) for i in own]
                      for x in (k, v)), st.pitch)
                want = (image & mask) | (0xA5 & ~mask)
                assert np.array_equal(pool[page_no, h, s], want), (page_no, h, s)
    # the other heads hold their own rows too
    got = st.read(i32(list(kept)))
    some = r.permutation(heads)[:24]
    for x, y in zip((k, v), got):
        want = np.stack([[O.row_values(*O.quantise_row(x[i, h])) for h in some]
                         for i in kept.values()])
        assert torch.equal(y.cpu()[:, some], torch.from_numpy(want).float().to(y.dtype))


def test_special_values(rba):
    p = Pair(rba, 9, heads=1, dim=128, page=16, dtype="f32", requests=1)
    k = rows(p.r, (8, 1, 128))
    k[0, 0, :32] = 0
    k[1, 0, 40] = np.inf
    k[2, 0, 70] = np.nan
    k[3, 0, 96:] = 2.0 ** -104          # below the least scale
    k[4, 0, :32] = 3.0e38               # near the largest
    k[5, 0, 32:64] = 0
    k[5, 0, 33] = 2.0 ** -95            # a lone small value keeps its scale
    k[6, 0] = -k[4, 0]
    k[7, 0, :32] = np.arange(-16, 16)   # halves: ties to even
    p.grow([8], pad=0, k=k, v=k[::-1].copy())
    got, v = p.st.read(i32(list(range(8))))
    want = np.stack([O.row_values(*O.quantise_row(x[0])) for x in k])
    np.testing.assert_array_equal(got[:, 0].cpu().numpy().astype(np.float64), want)
    np.testing.assert_array_equal(v[:, 0].cpu().numpy().astype(np.float64), want[::-1])
    assert np.isnan(want[1, 32:64]).all() and np.isfinite(want[1, :32]).all()


@pytest.mark.parametrize("heads,dim,page,tokens", [(1, 64, 1, 300), (3, 128, 2, 1000),
                                                   (40, 128, 17, 900), (2, 96, 33, 777),
                                                   (8, 64, 200, 5000)])
def test_means_of_every_page_that_a_call_completes(rba, heads, dim, page, tokens):
    """Few and many pages to a CTA, of one strip to thirteen; an open last page keeps its mean."""
    st = rba.PagedStore(n_q_heads=heads, n_kv_heads=heads, head_dim=dim, page_size=page,
                        n_pages=tokens // page + 2, max_requests=2, max_pages=tokens // page + 2)
    torch.manual_seed(page)
    slots = st.extend(i32([tokens // 3, tokens - tokens // 3]), tokens)[0]
    k = torch.randn((tokens, heads, dim), device="cuda").bfloat16()
    st.rep.fill_(7.0)
    st.append(slots, k, k)
    wide = rba.PagedStore(n_q_heads=heads, n_kv_heads=heads, head_dim=dim, page_size=page,
                          n_pages=st.n_pages, max_requests=2, max_pages=st.max_pages, dtype="f32",
                          pool=st.pool, rep=st.rep, table=st.table, lens=st.lens, free=st.free,
                          n_free=st.n_free)
    rows = wide.read(torch.arange(st.n_pages * page, dtype=torch.int32, device="cuda"))[0]
    rows = rows.view(st.n_pages, page, heads, dim).double()
    used = torch.zeros(st.n_pages, dtype=torch.bool)
    for r, n in enumerate((tokens // 3, tokens - tokens // 3)):
        used[st.table[r, :n // page].cpu().long()] = True
    want, got = rows.mean(1), st.rep[..., :dim].double()
    # page - 1 sums, each rounded to half a step of at most the sum of |x|; the products are exact,
    # the division adds one more
    tol = rows.abs().sum(1) * 2.0 ** -24 * (page + 1) / page
    assert ((got - want).abs()[used] <= tol[used]).all()
    assert (st.rep[~used] == 7.0).all()


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f32", 100), ("bf16", 36)])
def test_strided_rows(rba, dtype, dim):
    # slices of a fused projection, an odd head stride, a view that starts off a boundary
    heads, n = 2, 20
    p = Pair(rba, 4, heads=heads, dim=dim, dtype=dtype, requests=1)
    a, b, c = (rba.PagedStore(n_q_heads=4, n_kv_heads=heads, head_dim=dim, page_size=16,
                              n_pages=4, max_requests=1, max_pages=4, dtype=dtype)
               for _ in range(3))
    k, v = (cuda(rows(p.r, (n, heads, dim), dtype), dtype) for _ in range(2))
    slots = a.extend(i32([n]), n)[0]
    a.append(slots, k, v)
    fused = torch.zeros((n, 3, heads, dim), dtype=k.dtype, device="cuda")
    fused[:, 1], fused[:, 2] = k, v
    b.append(slots, fused[:, 1], fused[:, 2])
    odd = torch.zeros(n * heads * (dim + 1) + 1, dtype=k.dtype, device="cuda")
    kk = odd[1:].view(n, heads, dim + 1)[..., :dim]
    kk.copy_(k)
    c.append(slots, kk, v.flip(0).flip(0))
    assert torch.equal(a.pool, b.pool) and torch.equal(a.pool, c.pool)
    assert torch.equal(a.rep, b.rep) and torch.equal(a.rep, c.rep)


def test_slots_past_the_pool_are_flagged(rba):
    st = rba.PagedStore(n_q_heads=1, n_kv_heads=1, head_dim=64, page_size=4, n_pages=2,
                        max_requests=1, max_pages=2)
    x = torch.ones((3, 1, 64), device="cuda").bfloat16()
    st.append(i32([-1, 8, 2 ** 31 - 1]), x, x)
    assert not st.pool.any() and not st.rep.any()
    with pytest.raises(rba.RbaError):
        st.check()
    k, _ = st.read(i32([8, 0]))
    assert not k.any()
    with pytest.raises(rba.RbaError):
        st.check()


def test_empty_calls(rba):
    st = rba.PagedStore(n_q_heads=2, n_kv_heads=1, head_dim=64, page_size=4, n_pages=2,
                        max_requests=2, max_pages=2)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    slots, starts = st.extend(i32([0, 0]), 0)
    assert slots.numel() == 0 and starts.tolist() == [0, 0, 0]
    st.append(slots, e, e)
    assert st.read(slots)[0].shape == (0, 1, 64)
    q = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    idx = st.select(q, 3, 0, 0)
    assert (idx == -1).all()
    out, lse = st.attend(q, idx, 4, 4)
    assert not out.any() and torch.isneginf(lse).all()
    st.check()


# ---------------------------------------------------------------------------------------------
# selection

@pytest.mark.parametrize("heads,group,dim,page,dtype,lens,k,sink,window", [
    (2, 4, 128, 16, "bf16", [700, 0, 130, 47], 5, 16, 40),
    (1, 1, 64, 7, "f32", [400, 6, 7, 8], 3, 0, 0),
    (3, 2, 100, 50, "f32", [1049, 300], 6, 60, 33),
    (2, 16, 128, 8, "bf16", [600], 64, 4, 16),
    (1, 5, 96, 1, "f32", [200, 33], 17, 3, 9),
    (2, 1, 36, 24, "bf16", [24 * 30, 23, 24, 25], 40, 1000, 1)])
def test_selection_is_the_models(rba, heads, group, dim, page, dtype, lens, k, sink, window):
    p = Pair(rba, k, heads=heads, group=group, dim=dim, page=page, dtype=dtype,
             n_pages=sum(-(-n // page) for n in lens) + 1, requests=len(lens),
             columns=-(-max(lens) // page) + 2)
    p.grow(lens)
    # the definition starts from the stored means
    rep = p.st.rep.cpu().numpy().astype(np.float64)
    p.m.reps = {n: rep[n, :, :dim] for n in p.m.reps}
    q, qd = p.queries()
    got = p.st.select(qd, k, sink, window)
    p.st.check()
    assert np.array_equal(got.cpu().numpy(), p.m.select(q, k, sink, window))


def test_selection_ties_go_to_the_lower_page(rba):
    p = Pair(rba, 3, heads=1, group=1, dim=64, page=4, dtype="f32", requests=1, columns=40)
    p.grow([100])
    p.st.rep.copy_(torch.round(p.st.rep * 2))       # whole numbers: many equal scores
    p.st.rep[p.st.table[0, 5:9].long()] = p.st.rep[p.st.table[0, 20].long()].clone()
    p.m.reps = {n: p.st.rep[n, :, :64].cpu().numpy().astype(float) for n in p.m.reps}
    q = np.round(p.r.normal(size=(1, 1, 64)) * 2).astype(np.float32)
    for k in (1, 2, 3, 7, 24):
        got = p.st.select(cuda(q), k, 0, 0)
        assert np.array_equal(got.cpu().numpy(), p.m.select(q, k, 0, 0)), k


def test_a_candidate_between_sink_and_window(rba):
    """The window begins before the sink ends, in one page: a candidate, of no token of its own."""
    p = Pair(rba, 83, page=128, n_pages=4, requests=2, columns=3)
    p.grow([200, 100])
    q, qd = p.queries()
    assert p.m.parts(0, 100, 150) == (50, 50, [0])
    idx = p.st.select(qd, 2, 100, 150)
    assert idx.tolist() == [[[0, -1]] * 2, [[-1, -1]] * 2]
    p.same_attention(q, qd, idx.cpu().numpy(), 100, 150)


# ---------------------------------------------------------------------------------------------
# attention

ATTEND = [
    # heads, group, dim, page, dtype, lens, k, sink, window
    (2, 4, 128, 16, "bf16", [500, 1, 0, 130], 4, 16, 40),
    (2, 1, 128, 50, "bf16", [333, 49, 50, 51, 100], 2, 0, 21),
    (1, 2, 64, 64, "f32", [61], 0, 64, 128),
    (1, 8, 128, 16, "f32", [300, 17], 3, 5, 33),
    (2, 5, 100, 24, "f32", [200, 0, 25], 2, 30, 7),
    (1, 16, 128, 8, "bf16", [150, 9], 5, 3, 4),
    (1, 7, 36, 33, "f32", [400], 3, 50, 60),
    (1, 12, 64, 7, "bf16", [130, 64], 4, 0, 0),
    (3, 3, 96, 1, "f32", [70, 2], 9, 2, 5),
    (1, 4, 4, 16, "f32", [90], 2, 8, 16),
    (2, 4, 128, 128, "bf16", [1500, 127, 128], 3, 200, 100),
    (1, 4, 128, 16, "bf16", [16, 16, 16], 1, 0, 0),
    (1, 1, 128, 16, "f32", [40], 2, 0, 1),
    (1, 2, 64, 16, "bf16", [100, 3], 6, 2 ** 31 - 1, 2 ** 31 - 1),
]


def _attended(rba, seed, case):
    heads, group, dim, page, dtype, lens, k, sink, window = case
    p = Pair(rba, seed, heads=heads, group=group, dim=dim, page=page, dtype=dtype,
             n_pages=sum(-(-n // page) for n in lens) + 1, requests=len(lens),
             columns=-(-max(lens) // page) + 1)
    p.st.pool.fill_(0xFF)  # codes 15 and NaN scales wherever no row is written
    p.grow(lens)
    idx = None
    if k:
        idx = np.full((len(lens), heads, k), 2 ** 30)  # past the candidates: never read
        for r in range(len(lens)):
            cand = p.m.parts(r, sink, window)[2]
            for h in range(heads):
                pick = sorted(p.r.permutation(cand)[:k].astype(int))
                idx[r, h, :len(pick)] = pick
    return p, idx, sink, window


@pytest.mark.parametrize("case", ATTEND)
def test_attention_matches_the_oracle(rba, case):
    p, idx, sink, window = _attended(rba, 7, case)
    q, qd = p.queries()
    p.same_attention(q, qd, idx, sink, window)


@pytest.mark.parametrize("case", [ATTEND[0], ATTEND[3], ATTEND[6]])
def test_attention_over_all_tokens(rba, case):
    p, _, _, _ = _attended(rba, 8, case)
    q, qd = p.queries()
    ws = p.st.attend_workspace()
    a = p.same_attention(q, qd, None, 0, max(p.m.lens), workspace=ws)
    b = p.same_attention(q, qd, None, 0, 2 ** 31 - 1, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ws.fill_(0xFF)  # nothing is kept in a workspace
    c = p.same_attention(q, qd, None, 0, 2 ** 31 - 1, workspace=ws)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


@pytest.mark.parametrize("scale", [0.0, 1e-3, 3.0, -1.0])
def test_attention_scales(rba, scale):
    p, idx, sink, window = _attended(rba, 11, ATTEND[0])
    q, qd = p.queries()
    p.same_attention(q, qd, idx, sink, window, scale=scale)


@pytest.mark.parametrize("qs,ks,vs", [(2.0 ** -60, 2.0 ** 60, 1.0),
                                      (2.0 ** 60, 2.0 ** -60, 2.0 ** 100),
                                      (0.0, 1.0, 2.0 ** -90), (1.0, 0.0, 2.0 ** 60),
                                      (2.0 ** 10, 2.0 ** -10, 2.0 ** -60)])
def test_attention_ranges(rba, qs, ks, vs):
    p = Pair(rba, 13, heads=1, group=4, dim=128, requests=1, dtype="f32")
    k, v = (rows(p.r, (120, 1, 128)) * np.float32(x) for x in (ks, vs))
    p.grow([120], pad=0, k=k, v=v)
    q, qd = p.queries(qs)
    p.same_attention(q, qd, None, 0, 120)


def test_attention_value_scales_far_apart(rba):
    # rows of values from 2^-40 to 2^40 in one request, the large ones with small weights and late
    p = Pair(rba, 17, heads=1, group=4, dim=128, requests=1, dtype="f32", n_pages=64,
             columns=40)
    k, v = rows(p.r, (640, 1, 128)), rows(p.r, (640, 1, 128))
    v *= np.float32(2.0) ** np.linspace(-40, 40, 640).astype(np.float32)[:, None, None]
    p.grow([640], pad=0, k=k, v=v)
    q, qd = p.queries()
    p.same_attention(q, qd, None, 0, 640)
    p2 = Pair(rba, 17, heads=1, group=4, dim=128, requests=1, dtype="f32", n_pages=64,
             columns=40)
    p2.grow([640], pad=0, k=k[::-1].copy(), v=v[::-1].copy())
    p2.same_attention(q, qd, None, 0, 640)


def _terms_by_group(p, q, scale):
    """Of attention over all tokens of request 0, in fp64: (out [heads][group][dim], sum of weight x
    largest |v| of the row's 32 dims, the same shape, bound of the logits' error, strips)."""
    m, heads, D = p.m, p.heads, p.dim
    rows = [m.rows[m.tables[0][t // p.page] * p.page + t % p.page] for t in range(m.lens[0])]
    K, V = (np.stack([x[i] for x in rows], 1) for i in (0, 1))  # [heads][T][dim]
    Q = q[0].reshape(heads, -1, D).astype(np.float64)
    x = scale * np.einsum("hgd,htd->hgt", Q, K)
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    cuts = range(0, D, 32)
    top = lambda y: np.concatenate([np.repeat(np.abs(y[..., a:a + 32]).max(-1, keepdims=True),
                                              len(y[0, 0, a:a + 32]), -1) for a in cuts], -1)
    unit = max((scale * np.abs(Q) @ top(K).transpose(0, 2, 1)).max() * 15 / 7, np.abs(x).max())
    return (np.einsum("hgt,htd->hgd", w, V), np.einsum("hgt,htd->hgd", w, top(V)),
            24 * unit * 2.0 ** -24, m.lens[0] / 16 + 1)


def _same_by_group(p, q, qd):
    """Every output against its own terms: the tolerance of same_attention with the sum of a
    group's |terms| in the place of the largest |v| of all."""
    scale = p.dim ** -0.5
    out = p.st.attend(qd, None, 0, 2 ** 31 - 1, scale=scale)[0]
    p.st.check()
    ref, terms, dx, strips = _terms_by_group(p, q, scale)
    err = np.abs(out[0].cpu().numpy().reshape(ref.shape) - ref)
    tol = terms * (2 * dx + 8 * 2.0 ** -22 + strips * 2.0 ** -23)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


FORMS = [(4, 128, "f32"), (3, 128, "bf16"), (1, 64, "bf16"), (8, 100, "f32"), (5, 128, "bf16"),
         (12, 64, "f32")]


@pytest.mark.parametrize("group,dim,dtype", FORMS)
@pytest.mark.parametrize("apart", [24, 32, 40])
def test_attention_value_groups_far_apart(rba, group, dim, dtype, apart):
    """The groups of 32 dims have scales of their own: a small one loses nothing to a large one."""
    p = Pair(rba, 71, heads=2, group=group, dim=dim, requests=1, dtype=dtype, n_pages=64,
             columns=60)
    k, v = rows(p.r, (900, 2, dim), dtype), rows(p.r, (900, 2, dim), dtype)
    for g, a in enumerate(range(0, dim, 32)):
        v[:, 0, a:a + 32] *= np.float32(2.0 ** (-apart * (g % 2)))
        v[:, 1, a:a + 32] *= np.float32(2.0 ** (apart * (g % 3 - 1)))
    p.grow([900], pad=0, k=k, v=v)
    _same_by_group(p, *p.queries())


@pytest.mark.parametrize("group,dim,dtype", FORMS)
@pytest.mark.parametrize("where", [0, 450, 899])
def test_attention_huge_row_of_no_weight(rba, group, dim, dtype, where):
    """A row whose values are 2^40 times the others' with a weight of about 2^-90 and one of 2^30
    with about 2^-37: the other rows keep their bits."""
    p = Pair(rba, 73, heads=2, group=group, dim=dim, requests=1, dtype=dtype, n_pages=64,
             columns=60)
    k, v = (rows(p.r, (900, 2, dim), dtype) for _ in range(2))
    q = rows(p.r, (1, 2 * group, dim), dtype)
    q[..., 0], q[..., 1:32], k[..., 0] = 16.0, 0.0, 0.0
    for at, down, up in ((where, 62.0, 40), ((where + 100) % 900, 26.0, 30)):
        k[at] = 0
        k[at, :, 0] = -down * dim ** 0.5 / 16
        v[at] *= np.float32(2.0 ** up)
    if dtype == "bf16":
        k = bf16(k)
    p.grow([900], pad=0, k=k, v=v)
    _same_by_group(p, q, cuda(q, dtype))


@pytest.mark.parametrize("group,dim,dtype", FORMS)
@pytest.mark.parametrize("rising", [True, False])
def test_attention_weights_against_values(rba, group, dim, dtype, rising):
    """Weights that rise (fall) by 2^0.1 a row and values that fall (rise) by as much: every row's
    term counts alike, however far the reference and the scales have moved."""
    p = Pair(rba, 79, heads=2, group=group, dim=dim, requests=1, dtype=dtype, n_pages=64,
             columns=60)
    T = 900
    k, v = np.zeros((T, 2, dim), np.float32), rows(p.r, (T, 2, dim), dtype)
    q = rows(p.r, (1, 2 * group, dim), dtype)
    q[..., 0], q[..., 1:32] = 1.0, 0.0
    ramp = np.arange(T) if rising else np.arange(T)[::-1]
    k[:, :, 0] = (0.1 * math.log(2) * dim ** 0.5 * ramp)[:, None]
    v *= (2.0 ** (-0.1 * ramp + 45)).astype(np.float32)[:, None, None]
    if dtype == "bf16":
        k, v = bf16(k), bf16(v)
    p.grow([T], pad=0, k=k, v=v)
    _same_by_group(p, q, cuda(q, dtype))


@pytest.mark.parametrize("group,dim,dtype", FORMS)
@pytest.mark.parametrize("apart", [20, 28])
def test_attention_query_elements_far_apart(rba, group, dim, dtype, apart):
    """Small elements of q against large keys, large ones against small: logits to within what rba.h
    states, 2^-39 of a head's largest element an element beside the bound of same_attention."""
    p = Pair(rba, 89, heads=2, group=group, dim=dim, requests=1, dtype=dtype, n_pages=64,
             columns=60)
    k, q = rows(p.r, (300, 2, dim), dtype), rows(p.r, (1, 2 * group, dim), dtype)
    for g, a in enumerate(range(0, dim, 32)):
        by = np.float32(2.0 ** ((apart // 2) * (-1) ** g))
        q[..., a:a + 32] *= by
        k[..., a:a + 32] /= by
    p.grow([300], pad=0, k=k)
    qd = cuda(q, dtype)
    scale = dim ** -0.5
    out, lse = p.st.attend(qd, None, 0, 300, scale=scale)
    p.st.check()
    ref, rl, vmax, unit = p.m.attend(q, None, 0, 300, scale)
    held = np.stack([x[0] for x in p.m.rows.values()])
    most = max(np.abs(held[:, h]).sum(-1).max() * np.abs(q[0, h * group:(h + 1) * group]).max()
               for h in range(2))
    dx = 24 * unit * 2.0 ** -24 + scale * most * 2.0 ** -39
    tol = vmax * (2 * dx + 8 * 2.0 ** -22 + 20 * 2.0 ** -23)
    assert np.abs(out.cpu().numpy() - ref).max() <= tol
    assert np.abs(lse.cpu().numpy() - rl).max() <= dx + (np.abs(rl).max() + 4) * 2.0 ** -22


def test_attention_one_token_dominates(rba):
    p = Pair(rba, 19, heads=2, group=4, dim=64, requests=1, dtype="f32", n_pages=64,
             columns=40)
    q, qd = p.queries()
    k = rows(p.r, (500, 2, 64))
    k[311] = q[0].reshape(2, 4, 64).mean(1) * 20   # found late: the reference has to move
    k[20] = -k[311]
    p.grow([500], pad=0, k=k)
    p.same_attention(q, qd, None, 0, 500)


def test_values_that_are_not_finite_stay_in_their_place(rba):
    p = Pair(rba, 23, heads=2, group=2, dim=128, requests=2, dtype="f32")
    k, v = rows(p.r, (80, 2, 128)), rows(p.r, (80, 2, 128))
    v[10, 0, 40] = np.inf    # request 0, head 0, dims 32 .. 63
    k[70, 1, 0] = np.nan     # request 1, head 1
    p.grow([48, 32], pad=0, k=k, v=v)
    out = p.st.attend(p.queries()[1], None, 0, 80)[0].cpu().numpy()
    bad = np.zeros(out.shape, bool)
    bad[0, :2, 32:64] = True
    bad[1, 2:] = True
    assert np.array_equal(np.isnan(out), bad) and np.isfinite(out[~bad]).all()
    # outside the attended set they are not seen
    out, lse = p.st.attend(p.queries()[1], None, 4, 5)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("group,dim,dtype", FORMS)
def test_queries_that_are_not_finite_leave_other_heads_alone(rba, group, dim, dtype):
    p = Pair(rba, 101, heads=2, group=group, dim=dim, requests=2, dtype=dtype, n_pages=64,
             columns=60)
    p.grow([500, 37])
    q, qd = p.queries()
    bad = np.zeros(q.shape[:2], bool)
    for r, h, x in ((0, 0, np.nan), (0, 2 * group - 1, np.inf), (1, group, -np.inf)):
        qd[r, h, 5] = float(x)
        bad[r, h] = True
    out, lse = (x.cpu().numpy() for x in p.st.attend(qd, None, 4, 300, scale=dim ** -0.5))
    p.st.check()
    ref, rl, vmax, unit = p.m.attend(q, None, 4, 300, dim ** -0.5)
    dx = 24 * unit * 2.0 ** -24
    tol = vmax * (2 * dx + 8 * 2.0 ** -22 + 33 * 2.0 ** -23)
    assert np.abs(out - ref)[~bad].max(initial=0) <= tol
    assert np.abs(lse - rl)[~bad].max(initial=0) <= dx + (np.abs(rl).max() + 4) * 2.0 ** -22
    assert not np.isfinite(out[bad]).any()


def test_strided_queries(rba):
    p, idx, sink, window = _attended(rba, 29, ATTEND[0])
    q, qd = p.queries()
    wide = torch.zeros((qd.shape[0], 3, qd.shape[1], qd.shape[2] + 8), dtype=qd.dtype,
                       device="cuda")
    view = wide[:, 1, :, 3:3 + qd.shape[2]]
    view.copy_(qd)
    a, b = (p.st.attend(x, i32(idx), sink, window) for x in (qd, view))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(p.st.select(qd, 3, sink, window), p.st.select(view, 3, sink, window))


def test_bad_pages_and_lengths_are_skipped_and_flagged(rba):
    p, idx, sink, window = _attended(rba, 31, ATTEND[0])
    q, qd = p.queries()
    good = p.st.attend(qd, i32(idx), sink, window)[0].clone()
    p.st.check()
    bad = idx.copy()
    bad[0, 0, 1] = 999
    out = p.st.attend(qd, i32(bad), sink, window)[0]
    with pytest.raises(rba.RbaError):
        p.st.check()
    assert torch.equal(out[0, 4:], good[0, 4:]) and torch.isfinite(out).all()
    p.st.table[3, 0] = p.st.n_pages
    out = p.st.attend(qd, i32(idx), sink, window)[0]
    p.st.select(qd, 2, sink, window)
    with pytest.raises(rba.RbaError):
        p.st.check()
    assert torch.equal(out[0], good[0])
    p.st.lens[1] = 2 ** 30
    out = p.st.attend(qd, i32(idx), sink, window)[0]
    with pytest.raises(rba.RbaError):
        p.st.check()
    # (one strip fewer cuts the line of strips elsewhere: other partial sums)
    assert not out[1].any() and torch.allclose(out[0], good[0], rtol=0, atol=1e-4)


def test_python_refusals(rba):
    p = Pair(rba, 1)
    q = p.queries()[1]
    with pytest.raises(ValueError):
        p.st.attend(q.float(), None, 0, 8)
    with pytest.raises(ValueError):
        p.st.attend(q[..., ::2].repeat(1, 1, 2)[..., ::2], None, 0, 8)
    with pytest.raises(ValueError):
        p.st.attend(q, torch.zeros((3, 2, 1), dtype=torch.int64, device="cuda"), 0, 8)
    with pytest.raises(ValueError):
        p.st.attend(q.cpu(), None, 0, 8)
    with pytest.raises(ValueError):
        p.st.extend(i32([1, 2, 3]).cpu(), 6)
    with pytest.raises(ValueError):
        p.st.append(i32([0]), q[:1], q[:1])
    with pytest.raises(rba.RbaError):
        p.st.attend(torch.cat([q, q]), None, 0, 8)  # more requests than the table has rows
    with pytest.raises(rba.RbaError):
        p.st.attend(q, None, 0, 8, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        rba.PagedStore(n_q_heads=1, n_kv_heads=1, head_dim=64, page_size=8, n_pages=2,
                       max_requests=1, max_pages=2, lens=torch.zeros(2, dtype=torch.int32).cuda())


# ---------------------------------------------------------------------------------------------
# together

def test_decode_steps_replayed_while_requests_grow(rba):
    """One captured step (extend, append, select, attend) replayed over growing requests, one of
    them idle, with a request that ends and starts again; every step against the model."""
    requests, k, sink, window = 3, 2, 5, 20
    p = Pair(rba, 41, heads=2, group=4, dim=64, page=8, n_pages=60, requests=requests, columns=24)
    p.grow([70, 0, 33])
    st = p.st
    new = i32([1, 0, 1])
    slots = torch.empty(4, dtype=torch.int32, device="cuda")
    starts = torch.empty(requests + 1, dtype=torch.int32, device="cuda")
    kv = torch.zeros((4, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((requests, 8, 64), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((requests, 2, k), dtype=torch.int32, device="cuda")
    out, lse = (torch.empty((requests, 8, *d), device="cuda") for d in ((64,), ()))
    ws, sws = st.attend_workspace(), st.select_workspace()

    def step():
        st.extend(new, 4, slots=slots, starts=starts)
        st.append(slots, kv[:, 0], kv[:, 1])
        st.select(q, k, sink, window, idx=idx, workspace=sws)
        st.attend(q, idx, sink, window, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        saved = [t.clone() for t in (st.lens, st.n_free)]
        step()  # a first call of each kernel before the capture
        st.lens.copy_(saved[0])
        st.n_free.copy_(saved[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(30):
        grow = [1, int(i % 3 == 1), 1]
        if i == 17:
            st.truncate(i32([2 ** 31 - 1, 0, 40]))
            p.m.truncate([2 ** 31 - 1, 0, 40])
        new.copy_(i32(grow))
        k_new, v_new, qn = (rows(p.r, s, "bf16") for s in ((4, 2, 64), (4, 2, 64), (3, 8, 64)))
        kv.copy_(torch.stack([cuda(k_new), cuda(v_new)], 1))
        q.copy_(cuda(qn))
        graph.replay()
        st.check()
        want = p.m.extend(grow, 4)
        assert slots.tolist() == want + [-1] * (4 - len(want))
        p.m.append(want, k_new, v_new)
        rep = st.rep.cpu().numpy().astype(np.float64)
        p.m.reps = {n: rep[n] for n in p.m.reps}
        sel = p.m.select(qn, k, sink, window)
        assert np.array_equal(idx.cpu().numpy(), sel)
        ref, rl, vmax, unit = p.m.attend(qn, sel, sink, window, 64 ** -0.5)
        tol = vmax * (48 * unit * 2.0 ** -24 + 16 * 2.0 ** -22)
        assert np.abs(out.cpu().numpy() - ref).max() <= tol
        p.same_tables()


def test_readers_on_two_streams(rba):
    p, idx, sink, window = _attended(rba, 43, ATTEND[10])
    q, qd = p.queries()
    want = [t.clone() for t in p.st.attend(qd, i32(idx), sink, window)]
    sel = p.st.select(qd, 3, sink, window).clone()
    di = i32(idx)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [p.st.attend_workspace() for _ in streams]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append((*p.st.attend(qd, di, sink, window, workspace=w),
                            p.st.select(qd, 3, sink, window)))
    torch.cuda.synchronize()
    for out, lse, s in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(s, sel)


def test_decode_step_captured_and_replayed(rba):
    """The whole step in one graph with every buffer given, against the same calls made one by one on
    a second store, while requests grow, stay, end and start again."""
    a, b = (Pair(rba, 97, heads=2, group=4, dim=64, page=8, n_pages=60, columns=24)
            for _ in range(2))
    for p in (a, b):
        p.grow([70, 0, 33])
    st, k, sink, window = a.st, 3, 5, 20
    new = i32([0, 0, 0])
    kv = torch.zeros((4, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((3, 8, 64), dtype=torch.bfloat16, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    own = dict(slots=i32([0] * 4), starts=i32([0] * 4), idx=i32(np.zeros((3, 2, k))),
               out=torch.empty((3, 8, 64), **f32), lse=torch.empty((3, 8), **f32),
               select_workspace=st.select_workspace(), workspace=st.attend_workspace())

    def step():
        return st.decode_step(q, kv[:, 0], kv[:, 1], new, k, sink, window, **own)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # a first call of each kernel before the capture: no request grows
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    assert [t.data_ptr() for t in got] == [own[n].data_ptr() for n in ("idx", "out", "lse")]
    for i in range(24):
        grow = [1, int(i % 3 == 1), 2]
        if i == 13:
            for p in (a, b):
                p.st.truncate(i32([2 ** 31 - 1, 0, 40]))
        new.copy_(i32(grow))
        kv.copy_(torch.stack([cuda(rows(a.r, (4, 2, 64), "bf16")) for _ in range(2)], 1))
        q.copy_(cuda(rows(a.r, (3, 8, 64), "bf16")))
        graph.replay()
        slots, _ = b.st.extend(new, 4)
        b.st.append(slots, kv[:, 0], kv[:, 1])
        idx = b.st.select(q, k, sink, window)
        want = (idx, *b.st.attend(q, idx, sink, window))
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i
        assert torch.equal(own["slots"], slots) and torch.equal(st.lens, b.st.lens)
        assert torch.equal(st.pool, b.st.pool) and torch.equal(st.rep, b.st.rep)
        st.check()


def test_decode_step_is_the_four_calls(rba):
    a, b = (Pair(rba, 47, heads=2, group=2, dim=64, page=8, requests=3) for _ in range(2))
    for p in (a, b):
        p.grow([40, 0, 17])
    q, qd = a.queries()
    k, v = (cuda(rows(a.r, (5, 2, 64), "bf16"), "bf16") for _ in range(2))
    new = i32([1, 3, 0])
    got = a.st.decode_step(qd, k, v, new, 2, 4, 9)
    slots, _ = b.st.extend(new, 5)
    b.st.append(slots, k, v)
    idx = b.st.select(qd, 2, 4, 9)
    want = (idx, *b.st.attend(qd, idx, 4, 9))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(a.st.pool, b.st.pool) and a.st.lens.tolist() == [41, 3, 17]
    idx, out, lse = a.st.decode_step(qd, k[:0], v[:0], i32([0, 0, 0]), 0, 4, 9)
    assert idx is None and torch.isfinite(out).all()
    for bad in ((qd[:2], k, v, new), (qd, k[:4], v, new), (qd, k, v.float(), new),
                (qd, k, v, new.long())):
        with pytest.raises(ValueError):
            a.st.decode_step(*bad, 2, 4, 9)
    f32 = dict(dtype=torch.float32, device="cuda")
    for bad in (dict(idx=i32([[0]])), dict(out=torch.empty((3, 4, 32), **f32)),
                dict(lse=torch.empty((4, 3), **f32)), dict(slots=i32([0])),
                dict(starts=i32([0])), dict(workspace=torch.empty(64, **f32))):
        with pytest.raises(ValueError):
            a.st.decode_step(qd, k, v, new, 2, 4, 9, **bad)
    tiny = torch.empty(16, dtype=torch.uint8, device="cuda")
    for bad in (dict(select_workspace=tiny), dict(workspace=tiny)):
        with pytest.raises(rba.RbaError):
            a.st.decode_step(qd, k, v, new, 2, 4, 9, **bad)
    for bad in ((-1, 4, 9), (2, -1, 9), (2, 4, -1)):
        with pytest.raises(ValueError):
            a.st.decode_step(qd, k, v, new, *bad)
    assert a.st.lens.tolist() == [41, 3, 17]  # a refused step grows nothing
    a.st.check()


@pytest.mark.parametrize("shape,k,status", [
    (dict(heads=1, page=16, columns=20000), 3, 2),             # more candidates than select takes
    (dict(heads=256, page=16, columns=2 ** 20, requests=16), 0, 2)])  # a line attend cannot count
def test_a_step_that_the_library_refuses_grows_nothing(rba, shape, k, status):
    p = Pair(rba, 59, group=1, dim=64, n_pages=4, **shape)
    R = len(p.m.lens)
    q, x = p.queries()[1], torch.ones((1, p.heads, 64), device="cuda").bfloat16()
    new = i32([1] + [0] * (R - 1))
    before = [t.clone() for t in (p.st.lens, p.st.n_free, p.st.pool)]
    with pytest.raises(rba.RbaError) as e:
        p.st.decode_step(q, x, x, new, k, 0, 0)
    assert e.value.status == status
    assert all(torch.equal(a, b) for a, b in zip(before, (p.st.lens, p.st.n_free, p.st.pool)))
    p.st.check()


def test_a_step_with_a_workspace_off_its_boundary_grows_nothing(rba):
    p = Pair(rba, 61)
    q, x = p.queries()[1], torch.ones((1, 2, 128), device="cuda").bfloat16()
    wide = torch.empty(p.st.attend_workspace().numel() + 16, dtype=torch.uint8, device="cuda")
    for bad in (dict(workspace=wide[4:]), dict(select_workspace=wide[2:])):
        with pytest.raises(rba.RbaError) as e:
            p.st.decode_step(q, x, x, i32([1, 0, 0]), 2, 0, 0, **bad)
        assert e.value.status == rba.ERR_INVALID_ARG
        assert p.st.lens.tolist() == [0, 0, 0]


def test_numbers_past_32_bits_are_refused(rba):
    """As 32-bit numbers 2^32 is 0: attention without its window."""
    p = Pair(rba, 67)
    p.grow([9, 0, 30])
    q, qd = p.queries()
    x = torch.ones((1, 2, 128), device="cuda").bfloat16()
    for bad in ((2 ** 31, 0, 0), (0, 2 ** 32, 0), (0, 0, 2 ** 32), (0, 0, 2 ** 31)):
        with pytest.raises(ValueError):
            p.st.decode_step(qd, x, x, i32([1, 0, 0]), *bad)
        if not bad[0]:
            with pytest.raises(ValueError):
                p.st.attend(qd, None, *bad[1:])
            with pytest.raises(ValueError):
                p.st.select(qd, 1, *bad[1:])
    with pytest.raises(ValueError):
        p.st.extend(i32([1, 0, 0]), 2 ** 32 + 1, slots=i32([0]))
    with pytest.raises((TypeError, ValueError)):
        p.st.decode_step(qd, x, x, i32([1, 0, 0]), 0, 0, 30, scale="none")
    assert p.st.lens.tolist() == [9, 0, 30]
    a = p.st.decode_step(qd, x, x, i32([0, 0, 0]), 0, 0, 30, scale=np.float32(0.25))
    b = p.st.attend(qd, None, 0, 30, scale=0.25)
    assert torch.equal(a[1], b[0]) and torch.equal(a[2], b[1])


def test_tables_and_free_list_are_given_together(rba):
    """A free list made anew beside a table in use would hand out pages that requests hold."""
    sizes = dict(n_q_heads=2, n_kv_heads=2, head_dim=64, page_size=8, n_pages=6, max_requests=2,
                 max_pages=4)
    a = rba.PagedStore(**sizes)
    a.extend(i32([9, 8]), 17)
    own = dict(table=a.table, lens=a.lens, free=a.free, n_free=a.n_free)
    for take in range(1, 15):  # every choice but none and all
        with pytest.raises(ValueError):
            rba.PagedStore(**sizes, pool=a.pool,
                           **{n: t for i, (n, t) in enumerate(own.items()) if take >> i & 1})
    b = rba.PagedStore(**sizes, pool=a.pool, rep=a.rep, **own)
    slots = b.extend(i32([0, 16]), 16)[0]  # the pages that are left
    held = a.table[0, :2].tolist() + a.table[1, :3].tolist()
    assert len(set(held)) == 5 and a.lens.tolist() == [9, 24]
    assert not {s // 8 for s in slots.tolist()} & set(held[:2])
    c = rba.PagedStore(**sizes, pool=torch.zeros_like(a.pool))  # tables made for the memory given
    assert c.lens.tolist() == [0, 0] and int(c.n_free) == 6


def test_keys_that_are_not_finite_leave_other_rows_alone(rba):
    """A page mean that is not a number makes its own row's choice unspecified, no other's."""
    for k, columns in ((3, 24), (17, 80)):  # a warp's rows, a CTA's
        p = Pair(rba, 53, heads=2, group=2, dim=64, page=4, n_pages=120, requests=3,
                 columns=columns)
        keys = rows(p.r, (200, 2, 64), "bf16")
        keys[50, 1, 7], keys[130, 0, 3] = np.nan, np.inf  # request 0 head 1, request 1 head 0
        p.grow([90, 90, 20], pad=0, k=keys)
        q, qd = p.queries()
        got = p.st.select(qd, k, 0, 5).cpu().numpy()
        p.st.check()
        rep = p.st.rep.cpu().numpy().astype(np.float64)
        p.m.reps = {n: np.nan_to_num(rep[n]) for n in p.m.reps}
        want = p.m.select(q, k, 0, 5)
        for r in range(3):
            for h in range(2):
                if (r, h) in ((0, 1), (1, 0)):
                    assert len(set(got[r, h].tolist())) == k and (got[r, h] >= 0).all()
                    assert (got[r, h] < 22).all()
                else:
                    assert np.array_equal(got[r, h], want[r, h]), (k, r, h)


# lines of every kind: a unit cut over many CTAs; many short units to a CTA, more than it has
# warps; single warps with long lines; short units taken whole, more than the GPU has CTAs
LINES = [
    # heads, group, dim, dtype, lengths
    (2, 4, 128, "bf16", [19923, 77]),
    (4, 2, 64, "f32", [4000] + [16 + 5 * (i % 6) for i in range(300)]),
    (4, 2, 64, "f32", [760] + [16 + 5 * (i % 6) for i in range(300)]),
    (8, 4, 64, "bf16", [4500 - 13 * i for i in range(64)]),
    (32, 1, 64, "bf16", [48000]),
    (2, 8, 64, "f32", [90 + i % 40 for i in range(500)]),
    (1, 6, 100, "bf16", [700 + 31 * (i % 9) for i in range(40)] + [0, 1, 31, 32, 33]),
]


@pytest.mark.parametrize("case", LINES)
def test_lines_of_every_kind(rba, case):
    """Against torch in 64 bits on the rows as held (a 32-bit store on the same pool reads them:
    a bf16 read would round)."""
    heads, group, dim, dtype, lens = case
    r = np.random.default_rng(len(lens))
    n, page = sum(lens), 64
    shape = dict(n_q_heads=heads * group, n_kv_heads=heads, head_dim=dim, page_size=page,
                 n_pages=sum(-(-x // page) for x in lens), max_requests=len(lens),
                 max_pages=-(-max(lens) // page))
    st = rba.PagedStore(**shape, dtype=dtype)
    torch.manual_seed(len(lens))
    k, v = (torch.randn((n, heads, dim), device="cuda").to(st.tdtype) for _ in range(2))
    slots = st.extend(i32(lens), n)[0]
    st.append(slots, k, v)
    q = cuda(rows(r, (len(lens), heads * group, dim), dtype), dtype)
    ws = st.attend_workspace()
    out, lse = st.attend(q, None, 0, max(lens), workspace=ws)
    again = st.attend(q, None, 0, max(lens), workspace=ws)
    st.check()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    wide = rba.PagedStore(**shape, dtype="f32", pool=st.pool, rep=st.rep, table=st.table,
                          lens=st.lens, free=st.free, n_free=st.n_free)
    K, V = wide.read(slots)
    start = 0
    for i, T in enumerate(lens):
        if T == 0:
            assert not out[i].any() and torch.isneginf(lse[i]).all()
            continue
        Ki, Vi = (x[start:start + T].double() for x in (K, V))
        start += T
        Q = q[i].double().view(heads, group, dim)
        x = torch.einsum("hgd,thd->hgt", Q, Ki) * dim ** -0.5
        ref = torch.einsum("hgt,thd->hgd", x.softmax(-1), Vi).flatten(0, 1)
        unit = (Q.abs().sum(-1).max() * Ki.abs().max() * dim ** -0.5 * 15 / 7).item()
        # at most 32 strips are summed in the matrix unit at a time
        tol = Vi.abs().max().item() * (48 * unit * 2.0 ** -24 + 8 * 2.0 ** -22 + 32 * 2.0 ** -23)
        assert (out[i].double() - ref).abs().max().item() <= tol, i
        want = torch.logsumexp(x, -1).flatten()
        tol = 24 * unit * 2.0 ** -24 + (want.abs().max().item() + 4) * 2.0 ** -22
        assert (lse[i].double() - want).abs().max().item() <= tol, i


def test_offsets_past_32_bits(rba):
    """Pages past 4 GB of the pool and rows 2^31 elements apart: bit for bit what a small store on
    dense rows gives."""
    heads, page, D, n = 8, 128, 128, 700
    sizes = dict(n_q_heads=16, n_kv_heads=heads, head_dim=D, page_size=page, max_requests=2,
                 max_pages=8)
    many = 2 ** 32 // (heads * page // 16 * 2304) + 100
    def order(n_pages):
        return dict(table=torch.full((2, 8), -1, dtype=torch.int32, device="cuda"),
                    lens=i32([0, 0]), n_free=i32([n_pages]),
                    free=torch.arange(n_pages, dtype=torch.int32, device="cuda"))
    a = rba.PagedStore(**sizes, n_pages=many, **order(many))
    b = rba.PagedStore(**sizes, n_pages=8, **order(8))
    torch.manual_seed(3)
    k, v = (torch.randn((n, heads, D), device="cuda").bfloat16() for _ in range(2))
    far = torch.empty(2 ** 32 + 4 * heads * D, dtype=torch.bfloat16, device="cuda")
    kf, vf = (far.as_strided((3, heads, D), (2 ** 31, D, 1), at) for at in (0, heads * D))
    kf.copy_(k[-3:])
    vf.copy_(v[-3:])
    q = torch.randn((2, 16, D), device="cuda").bfloat16()
    qf = far.as_strided((2, 16, D), (2 ** 32, D, 1), 2 * heads * D)
    qf.copy_(q)
    got = []
    for st, rows, Q in ((a, ((k[:-3], v[:-3]), (kf, vf)), qf), (b, ((k, v),), q)):
        slots, _ = st.extend(i32([400, 300]), n)
        at = 0
        for x, y in rows:
            st.append(slots[at:at + len(x)], x, y)
            at += len(x)
        assert at == n and int(st.table[0, 0]) == st.n_pages - 1
        idx = st.select(Q, 1, 130, 100)
        got.append((idx, *st.attend(Q, idx, 130, 100), *st.read(slots)))
        st.check()
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert torch.equal(a.pool[-8:], b.pool) and torch.equal(a.rep[-8:], b.rep)
    assert not a.pool[:8].any()


@pytest.mark.parametrize("group,dtype", [(2, "bf16"), (8, "f32")])
def test_as_many_requests_as_a_table_holds(rba, group, dtype):
    """4096 requests of 0 to 71 tokens: select, attend and read against torch in 64 bits."""
    R, page, D, sink, window, k = 4096, 8, 64, 3, 20, 2
    shape = dict(n_q_heads=group, n_kv_heads=1, head_dim=D, page_size=page, n_pages=R * 9,
                 max_requests=R, max_pages=9)
    st = rba.PagedStore(**shape, dtype=dtype)
    torch.manual_seed(5)
    lens = torch.randint(0, 72, (R,), device="cuda").int()
    n = int(lens.sum())
    kv = torch.randn((n, 2, 1, D), device="cuda").to(st.tdtype)
    slots, starts = st.extend(lens, n)
    st.append(slots, kv[:, 0], kv[:, 1])
    q = torch.randn((R, group, D), device="cuda").to(st.tdtype)
    idx = st.select(q, k, sink, window)
    out, lse = st.attend(q, idx, sink, window)
    st.check()
    assert torch.equal(st.lens, lens) and int(starts[-1]) == n
    wide = rba.PagedStore(**shape, dtype="f32", pool=st.pool, rep=st.rep, table=st.table,
                          lens=st.lens, free=st.free, n_free=st.n_free)
    K, V = (torch.zeros((R, 72, D), dtype=torch.float64, device="cuda") for _ in range(2))
    r = torch.repeat_interleave(torch.arange(R, device="cuda"), lens.long())
    t = torch.arange(n, device="cuda") - starts[:-1].long()[r]
    for x, y in zip((K, V), wide.read(slots)):
        x[r, t] = y[:, 0].double()
    L, pos, j = lens.long()[:, None], torch.arange(72, device="cuda"), torch.arange(9, device="cuda")
    w0 = torch.minimum((L - window).clamp(min=0), L // page * page)
    cand = (j < L // page) & ((j + 1) * page > sink) & (j * page < w0)
    Q = q.double()
    score = torch.einsum("rd,rjd->rj", Q.sum(1), st.rep[st.table.long().clamp(min=0), 0, :D].double())
    score = score.float().masked_fill(~cand, -math.inf)
    best = score.sort(descending=True, stable=True).indices[:, :k]
    best = torch.where(torch.gather(cand, 1, best), best, 99).sort().values
    assert torch.equal(idx[:, 0].long(), torch.where(best == 99, -1, best))
    chosen = (best[:, :, None] == j).any(1)
    seen = (pos < L) & ((pos < torch.minimum(w0, torch.tensor(sink, device="cuda"))) | (pos >= w0) |
                        chosen.repeat_interleave(page, 1))
    x = (torch.einsum("rgd,rtd->rgt", Q, K) * D ** -0.5).masked_fill(~seen[:, None], -math.inf)
    some = seen.any(1)
    ref = torch.einsum("rgt,rtd->rgd", x.softmax(-1).nan_to_num(0.0), V)
    assert not out[~some].any() and torch.isneginf(lse[~some]).all() and (~some).any()
    unit = (Q.abs().sum(-1).max() * K.abs().max() * D ** -0.5 * 15 / 7).item()
    dx = 24 * unit * 2.0 ** -24
    tol = V.abs().max().item() * (2 * dx + 8 * 2.0 ** -22 + 6 * 2.0 ** -23)
    assert (out.double() - ref).abs().max().item() <= tol
    want = torch.logsumexp(x, -1)[some]
    assert (lse[some].double() - want).abs().max().item() <= dx + (
        want.abs().max().item() + 4) * 2.0 ** -22


@pytest.mark.parametrize("heads,group,page,k,requests", [(2, 1, 16, 3, 40), (1, 3, 8, 16, 9),
                                                         (1, 1, 4, 17, 5), (2, 2, 4, 64, 3)])
def test_selection_of_many_rows(rba, heads, group, page, k, requests):
    """Rows that one warp selects from and rows that a CTA does, ragged, against torch."""
    torch.manual_seed(k)
    lens = [(i * 977) % 3000 + i for i in range(requests)]
    columns = -(-max(lens) // page)
    st = rba.PagedStore(n_q_heads=heads * group, n_kv_heads=heads, head_dim=32, page_size=page,
                        n_pages=sum(-(-n // page) for n in lens) + 1, max_requests=requests,
                        max_pages=columns, dtype="f32")
    st.extend(i32(lens), sum(lens))
    st.rep[..., :32] = torch.randint(-3, 4, (st.n_pages, heads, 32), device="cuda").float()
    q = torch.randint(-2, 3, (requests, heads * group, 32), device="cuda").float()  # many ties
    got = st.select(q, k, 5, 33).cpu()
    st.check()
    Q = q.view(requests, heads, group, 32).sum(2).double().cpu()
    rep, table = st.rep[..., :32].double().cpu(), st.table.long().cpu()
    for i, T in enumerate(lens):
        full = T // page
        w0 = min(max(T - 33, 0), full * page)
        cand = torch.arange(5 // page, max(5 // page, min(full, -(-w0 // page))))
        for h in range(heads):
            s = rep[table[i, cand], h] @ Q[i, h]
            best = cand[s.sort(descending=True, stable=True).indices[:k]].sort().values
            want = torch.full((k,), -1)
            want[:len(best)] = best
            assert torch.equal(got[i, h].long(), want), (i, h)
