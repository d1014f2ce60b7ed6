"""Chunk attention where one CTA works through several units: short rows beside long ones, several row blocks per
head, against the plain 64-bit form and against each row called alone."""
import pytest
import torch

from tests.serving_helpers import check_spread, chunk_spread
from tests.test_gpu_serving import BF16, F16, F32, TAU, inputs, keys, paged_pair, rnd

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import kv_cache_compression_gear_b200 as gear


def ragged(H, prompts, dt, **codec):
    """A paged pair of these prompts, their values of the size of the keys so that the low-rank parts matter."""
    ppr = -(-max(prompts) // 64) + 1
    kc, vc = paged_pair(len(prompts), H, 64, sum(-(-n // 64) for n in prompts) + 4, ppr, 4, dt, **codec)
    by_length = {}
    for b, n in enumerate(prompts):
        by_length.setdefault(n, []).append(b)
    for n, rows in by_length.items():
        kc.encode_rows(rows, keys(n, len(rows), H, n, 128, dt=dt))
        vc.encode_rows(rows, keys(n + 1, len(rows), H, n, 128, dt=dt))
    return kc, vc


def check_rows(kc, vc, rows, counts, Hq, H, dt, alone):
    q, kn, vn = inputs(counts, Hq, H, dt)
    ref, sigma = chunk_spread(kc, vc, rows, counts, q, kn, vn, TAU)
    got = gear.chunk_attn(kc, vc, rows, counts, q, kn, vn, TAU, out_dtype=F32)
    check_spread(got, ref, sigma, F32)
    assert torch.equal(got, gear.chunk_attn(kc, vc, rows, counts, q, kn, vn, TAU, out_dtype=F32))
    at = 0
    for i, (b, n) in enumerate(zip(rows, counts)):
        if i in alone:
            s = slice(at, at + n)
            one = gear.chunk_attn(kc, vc, [b], [n], q[s], kn[s], vn[s], TAU, out_dtype=F32)
            check_spread(one, ref[s], sigma[s], F32, f"row {b} alone")
        at += n
    assert gear.device_status() == 0


LOW = dict(bits=2, group_size=64, outlier_frac=0.02, rank=8, buffer_rank=2)   # the low-rank part is a third of a key


@pytest.mark.parametrize("count,hq", [(1, 1), (4, 4), (17, 4)])   # few rows per unit, and more than 32
@pytest.mark.parametrize("dt", [F16, BF16])
def test_short_rows_before_long_ones(dt, count, hq):
    """Units of one tile, which one of the two softmax groups has no part in, followed by units of many in the same
    CTA: both groups take part in every hand-over of a unit's Rf, and none meets another unit's."""
    prompts = ([20, 33, 60, 41, 25, 50, 60, 20] * 2 + [3000, 2500]) * 3
    kc, vc = ragged(8, prompts, dt, **LOW)
    B = len(prompts)
    check_rows(kc, vc, range(B), [count] * B, 8 * hq, 8, dt, alone=(0, 3, 16, 17, B - 1))


def test_short_rows_without_prompts_between():
    """Rows whose units stage no Rf (never encoded) between rows that do."""
    prompts = [40, 60, 1500, 30, 2000, 61, 44, 900]
    kc, vc = ragged(8, prompts * 4, F16, **LOW)
    B = len(prompts) * 4
    for b in (1, 2, 5, 11, 17, 18, 30):
        kc.release_rows([b])
        vc.release_rows([b])
    check_rows(kc, vc, range(B), [3] * B, 16, 8, F16, alone=(0, 2, 4, 11))


@pytest.mark.parametrize("hq", [8, 16])   # three row blocks per head, and five, whose tiles are rebuilt ahead
@pytest.mark.parametrize("dt", [F16, BF16])
def test_row_blocks_of_one_tile(dt, hq):
    """Several row blocks of one tile each per head, many heads per CTA: the next head's Rf is staged only when all
    row blocks of the last head have read theirs."""
    B, H = 16, 16
    kc, vc = ragged(H, [16] * B, dt, **LOW)
    check_rows(kc, vc, range(B), [80] * B, H * hq, H, dt, alone=(0, 7, 15))


@pytest.mark.parametrize("at", [0, 13, 30])
def test_one_long_chunk_among_short_rows(at):
    """A call that is cut into launches so that the long chunk's tiles are rebuilt beside few others."""
    prompts = [2000 - 7 * b for b in range(31)]
    kc, vc = ragged(16, prompts, F16, **LOW)
    counts = [1] * 31
    counts[at] = 400
    check_rows(kc, vc, range(31), counts, 64, 16, F16, alone=(0, at, 30))


def test_refusals_name_their_reason():
    """The status of a refused call, not only that there is one."""
    from kv_cache_compression_gear_b200 import gear as G
    kc, vc = ragged(2, [40, 33], F16)
    q = rnd(1, 2, 2 * 129, 128)
    with pytest.raises(gear.GearError) as e:   # more than 128 query heads per kv head
        gear.chunk_attn(kc, vc, [0, 1], [1, 1], q, None, None, TAU)
    assert e.value.status == G.GEAR_ERR_UNSUPPORTED
    with pytest.raises(gear.GearError) as e:   # a row twice
        gear.chunk_attn(kc, vc, [1, 1], [1, 1], q[:, :4], None, None, TAU)
    assert e.value.status == G.GEAR_ERR_INVALID_ARG
    assert gear.chunk_attn(kc, vc, [0, 1], [0, 0], q[:0, :4], None, None, TAU).shape == (0, 4, 128)
