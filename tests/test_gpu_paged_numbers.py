"""Scores and values that are no numbers at VISIBLE positions of the paged attention: they reach the
row that sees them as they do in the formula (and in sal_attention_window), on each of the ways a
call can run: a cluster of one block or of several, pieces joined inside, pieces joined by a second
kernel."""
import pytest
import torch

from stream_ref import attend, attention_bound

pytestmark = pytest.mark.gpu

# lengths, heads, kv_heads, head_dim, page: which way the call runs
WAYS = {
    "cluster of one": ([120, 90, 40], 4, 2, 128, 16),
    "cluster of eight": ([1500, 700, 40], 4, 2, 64, 8),
    "joined inside": ([3000] * 20 + [17, 200], 4, 4, 128, 16),
    "joined by a kernel": ([9000, 5000, 33], 16, 2, 128, 32),
    "joined by a kernel, by its part": ([300] * 90, 40, 8, 64, 16),
}


def _api():
    from speech_audio_encoder_b200 import api
    return api


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _make(lengths, H, kvh, d, page):
    g = torch.Generator(device="cuda").manual_seed(H + page)
    counts = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(counts), generator=g, device="cuda").tolist()
    table, at = [], 0
    for c in counts:
        table.append(order[at:at + c] + [-1] * (max(counts) - c))
        at += c
    k, v = (torch.randn(1, sum(counts), kvh, page, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(len(lengths), H, d, generator=g, device="cuda").bfloat16()
    return _api().PagedCache(k, v, _ints(table), _ints(lengths)), q


def _place(cache, s, j):
    """(page, slot) of position j of sequence s."""
    page = cache.k.shape[3]
    return int(cache.table[s, j // page]), j % page


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("bad", ["q nan", "q inf", "k nan", "k inf", "v nan", "v inf"])
@pytest.mark.parametrize("at", [0, 37, -1])
def test_visible_values_that_are_no_numbers(way, bad, at):
    """One element of one head's query, key or value in row 0: every output that the formula takes
    through it is no finite number, all others are right, other rows and heads to the bit."""
    cache, q = _make(*WAYS[way])
    lengths, H, kvh, d, page = WAYS[way]
    clean = _api().sal_attention_paged(q, cache).clone().reshape(len(lengths), H, d)
    kind, value = bad.split()
    x, share = float(value), H // kvh
    p, slot = _place(cache, 0, at % lengths[0])
    h, e = kvh - 1, 5
    hit = torch.zeros(len(lengths), H, d, dtype=torch.bool, device="cuda")
    if kind == "q":
        q[0, H - 1, e] = x      # every score of that head is NaN or infinite, some of them +inf
        hit[0, H - 1] = True
    elif kind == "k":
        cache.k[0, p, h, slot, e] = x  # the score is NaN, or inf by the sign of the query
        hit[0, h * share:(h + 1) * share] = True if value == "nan" else (q[0, h * share:(h + 1) * share, e] > 0)[:, None]
    else:
        cache.v[0, p, h, slot, e] = x
        hit[0, h * share:(h + 1) * share, e] = True
    o = _api().sal_attention_paged(q, cache).reshape(clean.shape)
    assert not bool(torch.isfinite(o[hit]).any())
    if bad == "k inf":  # heads whose score for that key is -inf: a weight of zero, the rest is renormalised
        assert bool(torch.isfinite(o[~hit]).all())
        hit[0, h * share:(h + 1) * share] = True
    assert torch.equal(o[~hit], clean[~hit])
    # and the next call on clean inputs is not touched by it
    if kind == "q":
        q[0, H - 1, e] = 1.0
        assert bool(torch.isfinite(_api().sal_attention_paged(q, cache)).all())


@pytest.mark.parametrize("way", WAYS)
def test_a_row_without_keys_is_zeros_beside_one_that_is_no_number(way):
    cache, q = _make(*WAYS[way])
    q[0] = float("nan")
    cache.lengths[1] = 0
    o = _api().sal_attention_paged(q, cache)
    assert bool(torch.isnan(o[0]).all()) and not bool(o[1].any()) and bool(torch.isfinite(o[2:]).all())


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("which", ["the last", "the first sixteen", "every other sixteen", "all but one", "all"])
def test_scores_of_minus_infinity(way, which):
    """Visible keys whose score is -infinity have a weight of zero, also where a block of sixteen, a
    warp's or a piece's share of them has no other; where all of a row's are, the formula is 0 / 0."""
    lengths, H, kvh, d, page = WAYS[way]
    lengths = [lengths[0] + 1, *lengths[1:]]
    while lengths[0] % 16 != 1:  # the last key is alone in its block
        lengths[0] += 1
    cache, q = _make(lengths, H, kvh, d, page)
    clean = _api().sal_attention_paged(q, cache).reshape(len(lengths), H, d)
    q[0, :, 5] = 1.0
    n = lengths[0]
    j = torch.arange(n)
    off = {"the last": j == n - 1, "the first sixteen": j < 16, "every other sixteen": j // 16 % 2 == 0,
           "all but one": j != n // 2, "all": j >= 0}[which]
    at = torch.tensor([_place(cache, 0, x) for x in range(n)], device="cuda")
    lost = at[off.cuda()]
    cache.k[0, lost[:, 0], :, lost[:, 1], 5] = float("-inf")
    o = _api().sal_attention_paged(q, cache).reshape(clean.shape)
    assert torch.equal(o[1:], clean[1:])
    if which == "all":
        assert bool(torch.isnan(o[0]).all())
        return
    share = H // kvh
    for h in range(kvh):
        rows = slice(h * share, (h + 1) * share)
        ref, spread = attend(q[0, rows], cache.k[0, at[:, 0], h, at[:, 1]], cache.v[0, at[:, 0], h, at[:, 1]],
                             (~off).expand(share, n))
        over = (o[0, rows].double() - ref).abs() - attention_bound(ref, spread)
        assert float(over.max()) <= 0, (h, float(over.max()))
