"""Values that are no numbers in the windowed attention, seen and hidden ones in the same column, the
same tile and the same row: a row that hides one is summed again, a row that only sees some is
right as it is, and both are told apart key by key."""
import pytest
import torch

from stream_ref import attention_bound, visible, window_reference

pytestmark = pytest.mark.gpu

SHAPES = [
    # T, heads, kv_heads, head_dim, left, right, sinks, lengths
    (700, 10, 10, 128, -1, -1, 0, None), (700, 4, 4, 64, -1, 0, 0, [700, 433]), (1500, 4, 2, 128, 200, 0, 5, None),
    (1500, 40, 40, 64, 33, 70, 0, [1500, 1100]), (900, 20, 20, 128, 100, 3, 150, [900, 640]), (1100, 3, 3, 128, 300, 0, 37, None),
    (2000, 16, 4, 64, 90, 90, 20, None), (400, 2, 2, 128, 0, 0, 3, None), (640, 2, 2, 64, 128, 0, 16, [640, 129]),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(4))
def test_each_element_is_finite_where_all_that_its_row_sees_is(shape, seed):
    """Single elements of v at random keys (and at tiles' and windows' edges) become NaN or infinite,
    each in its own column: exactly the elements whose row sees one are no finite number, all
    others are right; seen infinities of one sign are that infinity."""
    from speech_audio_encoder_b200 import api
    T, H, kvh, d, left, right, sinks, lens = shape
    g = torch.Generator(device="cuda").manual_seed(seed + T)
    q, k, v = (torch.randn(2, h, T, d, generator=g, device="cuda").bfloat16() for h in (H, kvh, kvh))
    r = torch.Generator().manual_seed(seed)
    edges = [0, sinks, max(0, sinks - 1), 127, 128, 255, 256, T - 1, T - 2, (sinks | 15), T - 128]
    at = edges[seed::4] + torch.randint(0, T, (4,), generator=r).tolist()
    columns = torch.randperm(d, generator=r).tolist()
    kinds = [float("nan"), float("inf"), float("-inf")]
    placed = []
    for i, j in enumerate(at):
        h, x = i % kvh, kinds[(i + seed) % 3]
        v[0, h, j, columns[i]] = x
        placed.append((h, j, columns[i], x))
    lens = [T, T] if lens is None else lens
    o = api.sal_attention_window(q, k, v, left, right, sinks, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o = o.double().reshape(2, T, H, d)
    p, j = torch.arange(T)[:, None], torch.arange(T)[None, :]
    hit = torch.zeros(T, H, d, dtype=torch.bool, device="cuda")
    share = H // kvh
    seen = visible(p, j, lens[0], left, right, sinks).expand(T, T)
    for h, key, c, x in placed:
        rows = seen[:, key].cuda() & (torch.arange(T, device="cuda") < lens[0])
        heads = slice(h * share, (h + 1) * share)
        hit[rows, heads, c] = True
        if x == x:
            assert bool((o[0][rows][:, heads, c] == x).all()), (key, c)
        else:
            assert bool(torch.isnan(o[0][rows][:, heads, c]).all()), (key, c)
    ref, spread = window_reference(q, k, v, left, right, sinks, lens)
    for b, n in enumerate(lens):
        off = (o[b, :n] - ref[b, :n]).abs() - attention_bound(ref[b, :n], spread[b, :n])
        assert bool((off[~hit[:n]] <= 0).all()) if b == 0 else float(off.max()) <= 0


@pytest.mark.parametrize("left,right", [(-1, -1), (-1, 0), (300, 300)])
def test_an_infinite_value_beside_hidden_ones_in_its_column(left, right):
    """One column: infinite at one key, NaN at others. A row that sees the infinity alone gives it."""
    from speech_audio_encoder_b200 import api
    T, H, d = 1300, 3, 128
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn(1, H, T, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    v[0, :, 100, 9] = float("inf")
    for key in (420, 421, 700, 1299):
        v[0, :, key, 9] = float("nan")
    o = api.sal_attention_window(q, k, v, left, right).double().reshape(T, H, d)
    p, j = torch.arange(T)[:, None], torch.arange(T)[None, :]
    seen = visible(p, j, T, left, right, 0).expand(T, T).cuda()
    nan = seen[:, [420, 421, 700, 1299]].any(1)
    inf = seen[:, 100] & ~nan
    assert bool(torch.isnan(o[nan][:, :, 9]).all()) and bool((o[inf][:, :, 9] == float("inf")).all())
    assert bool(torch.isfinite(o[~(nan | inf)]).all()) and bool(torch.isfinite(o[:, :, :9]).all())
