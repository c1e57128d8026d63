"""Pins of the oracle's paged 4-bit memory against things other than itself: torch's bf16
rounding and fp64 attention, closed forms of the quantisation, the layout read back bit by bit,
and brute force over the page tables."""
import math

import numpy as np
import pytest
import torch

import oracle as O


def test_bf16_rounding_is_torchs():
    x = np.random.default_rng(0).normal(size=4096).astype(np.float32) * \
        np.float32(2.0) ** np.random.default_rng(1).integers(-60, 60, 4096).astype(np.float32)
    ties = (np.arange(256, dtype=np.uint32) << 16 | 0x3F808000).view(np.float32)
    for v in (x, ties, np.array([0, -0.0, np.inf, -np.inf], np.float32)):
        assert np.array_equal(O.round_bf16(v), torch.from_numpy(v).bfloat16().float().numpy())


def test_quantise_closed_forms():
    # a ramp of whole steps is held exactly: largest 7, scale 1
    row = np.array([c for c in range(-7, 8)] + [0] * 17, np.float32)
    codes, s = O.quantise_row(row)
    assert s.tolist() == [1.0] and np.array_equal(O.row_values(codes, s), row.astype(float))
    # half-way values go to the even code
    codes, _ = O.quantise_row(np.array([7, 0.5, 1.5, 2.5, -0.5, -1.5] + [0] * 26, np.float32))
    assert codes[:6].tolist() == [7, 0, 2, 2, 0, -2]
    # zeros, tiny groups and groups that are not finite; the neighbour keeps its own scale
    row = np.concatenate([np.zeros(32), np.full(32, 2.0 ** -110), np.full(32, 3.0),
                          np.full(4, np.inf)]).astype(np.float32)
    codes, s = O.quantise_row(row)
    assert s[0] == 0 and s[1] == 0 and np.isnan(s[3]) and not codes[:64].any()
    assert np.abs(O.row_values(codes, s)[64:96] - 3.0).max() <= 3.0 * 2.0 ** -8
    # error within half a step (and the scale's own rounding) everywhere
    x = np.random.default_rng(2).normal(size=(50, 128)).astype(np.float32)
    for row in x:
        codes, s = O.quantise_row(row)
        assert (np.abs(O.row_values(codes, s) - row) <=
                np.repeat(s, 32) * (0.5 + 7 * 2.0 ** -8)).all()


@pytest.mark.parametrize("P,D", [(128, 128), (128, 100), (64, 64), (64, 36)])
def test_strip_image_read_back(P, D):
    r = np.random.default_rng(P + D)
    G = P // 32
    rows = [[O.quantise_row(r.normal(size=D).astype(np.float32)) for _ in range(16)]
            for _ in range(2)]
    image, mask = O.strip_image(rows[0], rows[1], P)
    assert (mask == 255).all() and len(image) == 16 * P + 64 * G
    units = image.view(np.uint16)
    for t in range(16):
        for d in range(D):
            # K: words of 8 dims in the order [token][c][group]; V: token pairs side by side
            word = image.view(np.uint32)[(t * 4 + d // 8 % 4) * G + d // 32]
            assert (word >> (4 * (d % 8))) & 15 == rows[0][t][0][d] + 8
            unit = units[4 * P + (((t // 8 * 8 + d // 4 % 8) * 4 + t // 2 % 4) * G + d // 32) * 2
                         + t % 2]
            assert (unit >> (4 * (d % 4))) & 15 == rows[1][t][0][d] + 8
    scales = (units[8 * P:].astype(np.uint32) << 16).view(np.float32).reshape(16, 2, G)
    for which in (0, 1):
        for t in range(16):
            assert np.array_equal(scales[t, which, :len(rows[which][t][1])], rows[which][t][1])


def test_tables_grow_and_shrink():
    m = O.PagedModel(1, 4, 3, 10, 3, 4)
    assert m.extend([4, 0, 1], 8) == [0, 1, 2, 3, 6]
    assert m.tables == [[0, 1], [], [2]] and m.free[::-1][:2] == [3, 4]
    before = list(m.free)
    assert m.extend([2, 7, 0], 9) == [4, 5, 9, 10, 11, 12, 13, 14, 15]
    m.truncate([4, 0, 1])
    assert m.free == before and m.tables == [[0, 1], [], [2]] and m.lens == [4, 0, 1]
    assert m.extend([9, 0, 0], 9) is None and m.extend([0, 2, 0], 1) is None
    assert m.extend([8, 12, 12], 40) is None and m.lens == [4, 0, 1]
    m.truncate([0, 0, 0])
    assert sorted(m.free) == list(range(10))


def _filled(seed, page=5, lens=(23, 0, 11), heads=2, dim=40):
    r = np.random.default_rng(seed)
    m = O.PagedModel(heads, dim, page, 40, len(lens), 12)
    slots = m.extend(list(lens), sum(lens))
    k, v = (r.normal(size=(sum(lens), heads, dim)).astype(np.float32) for _ in range(2))
    m.append(slots, k, v)
    return m, r


def test_attend_all_tokens_is_dense_attention():
    m, r = _filled(3)
    q = r.normal(size=(3, 4, 40)).astype(np.float32)
    out, lse, _, _ = m.attend(q, None, 0, 99, 0.3)
    for i, T in enumerate(m.lens):
        if T == 0:
            assert not out[i].any() and np.isneginf(lse[i]).all()
            continue
        K, V = (np.stack([m.rows[m.tables[i][t // 5] * 5 + t % 5][w] for t in range(T)])
                for w in (0, 1))
        for hq in range(4):
            want = torch.nn.functional.scaled_dot_product_attention(
                *(torch.from_numpy(np.ascontiguousarray(x))[None, None]
                  for x in (q[i, hq].astype(float)[None], K[:, hq // 2], V[:, hq // 2])),
                scale=0.3)
            assert np.abs(want.numpy()[0, 0, 0] - out[i, hq]).max() < 1e-12
            assert abs(np.log(np.exp(0.3 * K[:, hq // 2] @ q[i, hq]).sum()) - lse[i, hq]) < 1e-12


def test_every_candidate_selected_is_dense_attention():
    m, r = _filled(4)
    q = r.normal(size=(3, 4, 40)).astype(np.float32)
    idx = m.select(q, 9, 2, 3)
    assert idx[0, 0].tolist() == [0, 1, 2, 3] + [-1] * 5 and (idx[1] == -1).all()
    for a, b in zip(m.attend(q, idx, 2, 3, 0.3)[:2], m.attend(q, None, 0, 99, 0.3)[:2]):
        assert np.allclose(a, b, atol=1e-12)


def test_selection_by_rank_counting_and_ties():
    m, r = _filled(5, lens=(53, 8))
    for p in m.reps:  # pages come in equal pairs: the lower page of a request wins
        m.reps[p] = np.round(m.reps[p] * 2)
    m.reps[m.tables[0][7]] = m.reps[m.tables[0][2]].copy()
    q = np.round(r.normal(size=(2, 2, 40))).astype(np.float32)
    idx = m.select(q, 3, 0, 5)
    for h in range(2):
        s = [float(q[0, h] @ m.reps[p][h]) for p in m.tables[0][:10]]
        rank = [sum(x > s[j] or (x == s[j] and i < j) for i, x in enumerate(s))
                for j in range(10)]
        assert idx[0, h].tolist() == [j for j in range(10) if rank[j] < 3]


@pytest.mark.parametrize("T,page,sink,window", [(23, 5, 0, 0), (23, 5, 4, 7), (20, 5, 30, 2),
                                                (4, 5, 0, 1), (1, 1, 0, 0), (23, 5, 2, 99)])
def test_parts_partition_the_request(T, page, sink, window):
    m = O.PagedModel(1, 4, page, 40, 1, 30)
    m.extend([T], T)
    end, w0, cand = m.parts(0, sink, window)
    assert w0 <= max(T - window, 0) and (T - w0 >= T % page)
    inner = {t for j in cand for t in range(j * page, (j + 1) * page) if end <= t < w0}
    assert inner == set(range(end, w0))
    assert all((j + 1) * page <= T for j in cand)
