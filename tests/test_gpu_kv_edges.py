"""The 8-bit key/value cache where sizes differ most: rows beside much larger ones,
many sequences, long ones.  Against plain 64-bit arithmetic (kv_reference.py), as in
test_gpu_kv.py.
"""
import pytest
import torch

from kv_reference import out_bound, read_cache
from test_gpu_kv import Pair, score_bound

pytestmark = pytest.mark.gpu


def append(p, counts, edit):
    """Rows of each sequence, edited by edit(k or v, on the CPU); into both caches."""
    (_, k, v), start = p.rows(counts)
    for x in (k, v):
        edit(x[0])
        x[1].copy_(x[0])
    p.c.append(k[1], v[1], start, p.len, max(counts))
    p.len += torch.tensor(counts, dtype=torch.int32, device="cuda")
    first = 0
    for b, r in enumerate(counts):
        p.ref.append(b, k[0][first:first + r], v[0][first:first + r])
        first += r


def scores(p, of):
    """The score of every token held: of(b, h, n) gives a head's."""
    for b, n in enumerate(p.len.tolist()):
        pg = p.c.page_table[b, :-(-n // 64)].long()
        for h in range(p.heads):
            x = torch.zeros(len(pg) * 64)
            x[:n] = of(b, h, n)
            p.c.score[pg, h] = x.view(-1, 64).cuda()
    p.ref.score = read_cache(p.c, p.len.tolist())[2]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("large", [10, 13, 16, 18])
@pytest.mark.parametrize("stays", [False, True])
def test_evict_rows_that_leave_a_much_larger_one(gsi, fmt, dim, large, stays):
    """One row of each page is 2^large times the others and sets their scale.  It is
    evicted, or lands in another block than some of them; a page of zeros among them."""
    p = Pair(gsi, 2, 2, 1, dim, fmt, max_pages=8, spare=5, seed=large + dim)
    counts = [320, 300]

    def at(page, h):
        return 64 * page + (11 * page + 29 * h + 7) % 64

    def edit(x):
        for first in (0, 320):
            x[first + 64:first + 128] = 0
            for h in range(2):
                for page in range(5):
                    if first + at(page, h) < 620:
                        row = x[first + at(page, h), h * dim:(h + 1) * dim]
                        row.copy_(torch.randn(dim, generator=p.gen) * 2.0 ** large)

    append(p, counts, edit)
    p.check_cache()

    def of(b, h, n):
        s = torch.rand(n, generator=p.gen)
        for page in range(-(-n // 64)):
            if at(page, h) < n:
                s[at(page, h)] = 2.0 if stays else -1.0
        return s

    scores(p, of)
    for budget, recent in ((256, 0), (192, 5), (130, 60)):
        p.c.evict(p.len, budget, recent, p.spare)
        for b in range(2):
            p.ref.evict(b, budget, recent)
        p.check_cache(0.0)
    assert p.c.status() == 0
    p.c.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_evict_least_codes(gsi, fmt, dim):
    """Rows of a page's few least codes, alone in their new block: its scale is finer
    by the greatest factor that there is (2^17 for e4m3, whose least code is 2^-9)."""
    low = 1.0 if fmt == "int8" else 2.0 ** -9
    for few in (1, 2, 3, 4, 7):
        p = Pair(gsi, 1, 1, 1, dim, fmt, max_pages=4, spare=2, seed=few)

        def edit(x):
            x.copy_(torch.randint(-few, few + 1, x.shape, generator=p.gen) * low)
            x[::2, 3] = few * low
            x[5, 9] = x[64 + 60, 0] = 127.0 if fmt == "int8" else 448.0

        append(p, [128], edit)
        scores(p, lambda b, h, n: torch.tensor([-1.0 if t in (5, 124) or t % 2 else 1.0 for t in range(n)]))
        p.c.evict(p.len, 64, 0, p.spare)
        p.ref.evict(0, 64, 0)
        # the even rows but 124, and of the others the first: neither 5 nor 124
        assert p.ref.k[0][0].abs().max() <= few * low
        p.check_cache(0.0)
        p.c.close()

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,group", [(1, 1), (1, 8), (3, 4), (40, 2), (150, 1)])
@pytest.mark.parametrize("lse", [True, False])
def test_attention_over_values_of_all_sizes(gsi, dim, rows, group, lse):
    """Blocks whose values differ by up to 2^170: a row's divisor counts them alike,
    whichever comes first, in one share of a head or in several."""
    for sizes in ((90, None, 0, 85), (None, 90), (-70, 40, -70, 89, 0, -70), (0, None, None, 90, None, 3)):
        p = Pair(gsi, 2, 1, group, dim, "int8", max_pages=16, seed=rows + dim)
        n = 64 * len(sizes)

        def edit(x):
            for first in (0, n):
                for j, size in enumerate(sizes):
                    x[first + 64 * j:first + 64 * j + 64] *= 0.0 if size is None else 2.0 ** size

        (_, k, v), start = p.rows([n, n])
        edit(v[0])
        v[1].copy_(v[0])
        p.c.append(k[1], v[1], start, p.len, n)
        p.len += n
        for b in range(2):
            p.ref.append(b, k[0][b * n:b * n + n], v[0][b * n:b * n + n])
        p.check_out([rows, 1], lse=lse, accumulate=lse)
        assert p.c.status() == 0
        p.c.close()


def test_a_bound_of_rows_above_the_rows_of_a_call(gsi):
    """A fixed bound, say of drafted tokens, with fewer new rows in all, and with none."""
    p = Pair(gsi, 3, 2, 2, 64, "int8", seed=23)
    p.step([70, 1, 130])
    for counts in ([1, 0, 2], [0, 1, 0], [0, 0, 0]):
        (q, k, v), start = p.rows(counts)
        p.c.append(k[1], v[1], start, p.len, 5)
        out = p.c.attention(q[1], start, p.len, 5, accumulate=True)
        p.len += torch.tensor(counts, dtype=torch.int32, device="cuda")
        first = 0
        for b, r in enumerate(counts):
            if r:
                rows = slice(first, first + r)
                p.ref.append(b, k[0][rows], v[0][rows])
                ro, _, mag, absv = p.ref.attend(b, q[0][rows], 64 ** -0.5)
                assert ((out[rows].cpu().double() - ro).abs() <= out_bound(ro, mag, absv)).all()
            first += r
        p.check_cache()
    assert p.c.status() == 0
    p.c.close()


@pytest.mark.parametrize("seqs,heads,group,dim,rows", [(33, 2, 1, 64, 1), (100, 1, 4, 128, 3), (100, 2, 3, 256, 2),
                                                       (1100, 2, 1, 64, 1), (1100, 1, 5, 64, 2)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_attention_of_few_rows_of_many_sequences(gsi, seqs, heads, group, dim, rows, accumulate):
    """More sequences than a warp has lanes, and than shared memory counts at once;
    runs of sequences without new rows over their edges."""
    p = Pair(gsi, seqs, heads, group, dim, "e4m3", max_pages=3, seed=seqs + dim)
    first = torch.randint(0, 140, (seqs,), generator=p.gen).tolist()
    first[0], first[seqs - 1] = 0, 129
    p.step(first, lse=False)
    mag, sums = 0.0, 0
    for gap in ((30, 66), (1, 32), (seqs - 80, seqs - 1), (seqs, seqs)):
        counts = torch.randint(0, rows + 1, (seqs,), generator=p.gen).tolist()
        counts[0] = counts[seqs - 1] = rows
        for b in range(max(gap[0], 1), min(gap[1], seqs - 1)):
            counts[b] = 0
        mag = max(mag, p.check_out(counts, accumulate=accumulate, lse=accumulate))
        sums += rows * group
    assert p.c.status() == 0
    p.check_cache(score_bound(mag, sums) if accumulate else None)
    p.c.close()


@pytest.mark.parametrize("tokens,budget,recent", [(46000, 1000, 100), (46000, 45500, 200), (262400, 20000, 64)])
def test_evict_from_long_sequences(gsi, tokens, budget, recent):
    """More scores, and more pages, than the selection keeps in shared memory."""
    own, spare = -(-tokens // 64), -(-budget // 64)
    p = Pair(gsi, 1, 1, 1, 64, "e4m3", max_pages=own, spare=spare, seed=budget)
    append(p, [tokens], lambda x: None)
    scores(p, lambda b, h, n: torch.floor(300 * torch.rand(n, generator=p.gen) ** 3))
    p.c.evict(p.len, budget, recent, p.spare)
    p.ref.evict(0, budget, recent)
    p.check_cache(0.0)
    assert p.c.status() == 0
    p.c.close()
