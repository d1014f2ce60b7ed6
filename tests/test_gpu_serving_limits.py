"""Chunk attention within the statistical limit of its roundings (a few thousandths of a row's norm in ordinary
ranges), over the types, codecs, layouts and lengths of the bound's tests."""
import pytest
import torch

from tests.serving_helpers import check_spread, chunk_spread
from tests.test_gpu_serving import (BF16, CHUNK, F16, F32, REBUILT, TAU, encode, inputs, keys, make, paged_pair, rnd)

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import kv_cache_compression_gear_b200 as gear


@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("rows,case", [([2, 0, 1], c) for c in CHUNK] + [([1, 2, 0], c) for c in REBUILT])
def test_chunk_attn_within_its_roundings(rows, case, own):
    dt, H, hq, P, prompts, appended, counts, codec = case
    kc, vc = make(dt, H, P, prompts, appended, codec)
    q, kn, vn = inputs(counts, H * hq, H, dt)
    if not own:
        kn = vn = None
    ref, sigma = chunk_spread(kc, vc, rows, counts, q, kn, vn, TAU)
    for od in (F32, dt):
        check_spread(gear.chunk_attn(kc, vc, rows, counts, q, kn, vn, TAU, out_dtype=od), ref, sigma, od)
    assert gear.device_status() == 0


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("B,n,count", [(1, 20000, 3), (2, 9000, 40), (1, 20000, 700), (200, 40, 2)])
def test_long_contexts_within_their_roundings(dt, B, n, count):
    """Units cut over many CTAs, more sequences than a launch holds."""
    kc, vc = paged_pair(B, 2, 64, B * (n // 64 + 2), n // 64 + 2, 4, dt)
    kc.encode_rows(range(B), rnd(3, B, 2, n, 128, dt=dt))
    vc.encode_rows(range(B), keys(4, B, 2, n, 128, dt=dt))
    q, kn, vn = inputs([count] * B, 4, 2, dt)
    ref, sigma = chunk_spread(kc, vc, range(B), [count] * B, q, kn, vn, TAU)
    check_spread(gear.chunk_attn(kc, vc, range(B), [count] * B, q, kn, vn, TAU, out_dtype=F32), ref, sigma, F32)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("counts", [[3, 1, 2], [40, 33, 1], [700, 5, 64]])
def test_caches_grown_by_appends(dt, counts):
    """Rows of which most tokens were flushed in blocks of 20, each with a low-rank factor of its own."""
    kc, vc = paged_pair(3, 2, 64, 60, 20, 64, dt, rank=4, buffer_rank=4, bits=2, group_size=32)
    encode(kc, vc, [0, 1, 2], 17, 4, dt)
    new = [1000, 431, 20]
    T = sum(new)
    gear.append_rope_rows(kc, vc, range(3), new, keys(7, T, 2, 128, dt=dt), keys(8, T, 2, 128, dt=dt))
    assert kc.counters()[1].tolist() == [1 + 49, 1 + 21, 1]
    q, kn, vn = inputs(counts, 8, 2, dt)
    ref, sigma = chunk_spread(kc, vc, range(3), counts, q, kn, vn, TAU)
    check_spread(gear.chunk_attn(kc, vc, range(3), counts, q, kn, vn, TAU, out_dtype=F32), ref, sigma, F32)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("counts", [[2, 1, 8, 4], [300, 1, 270, 1600]])
def test_padded_prompts_within_their_roundings(dt, counts):
    p = gear.make_params(rank=7, buffer_rank=3, outlier_frac=0.05)
    kc, vc = gear.Cache(p, 4, 2, 300, 2, dt), gear.Cache(p, 4, 2, 300, 2, dt)
    kc.encode(keys(1, 4, 2, 260, 128, dt=dt))
    vc.encode(rnd(2, 4, 2, 260, 128, dt=dt))
    plen = torch.tensor([260, 130, 0, 31], dtype=torch.int32, device="cuda")
    q, kn, vn = inputs(counts, 4, 2, dt)
    ref, sigma = chunk_spread(kc, vc, range(4), counts, q, kn, vn, TAU, plen=plen.tolist())
    got = gear.chunk_attn(kc, vc, range(4), counts, q, kn, vn, TAU, prefill_len=plen, out_dtype=F32)
    check_spread(got, ref, sigma, F32)


def test_shared_heads_and_single_tokens_agree_with_decode():
    """One token per row: chunk attention within its limit, decode attention (binary32) far within it."""
    kc, vc = make(F16, 4, 64, [3000, 77, 1300], [33, 20, 5], dict())
    q = rnd(9, 3, 16, 128)
    ref, sigma = chunk_spread(kc, vc, [0, 1, 2], [1, 1, 1], q, None, None, TAU)
    check_spread(gear.chunk_attn(kc, vc, [0, 1, 2], [1, 1, 1], q, None, None, TAU, out_dtype=F32), ref, sigma, F32)
    check_spread(gear.decode_attn(kc, vc, q, TAU, out_dtype=F32), ref, sigma / 4, F32)
