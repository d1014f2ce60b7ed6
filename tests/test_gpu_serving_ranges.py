"""Chunk attention over values and queries of very different size, in every kernel: few query rows per unit, some,
paired row tiles, tiles rebuilt ahead."""
import math

import pytest
import torch

from tests.serving_helpers import check_chunk, check_spread, chunk_ref, chunk_spread
from tests.test_gpu_serving import BF16, F16, F32, TAU, keys, paged_pair, rnd

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import kv_cache_compression_gear_b200 as gear

COUNTS = [3, 30, 60, 300]   # with four query heads: 12, 120, 240 and 1200 rows


def pair(n, dt, k, v, pages=64, **codec):
    """A paged pair of one sequence, keys and values [H][n][128] given."""
    kc, vc = paged_pair(1, k.shape[0], pages, -(-n // pages) + 2, -(-n // pages) + 2, 4, dt, **codec)
    kc.encode_rows([0], k[None].to(dt).contiguous())
    vc.encode_rows([0], v[None].to(dt).contiguous())
    return kc, vc


def check(kc, vc, q, kn, vn, tau, what=""):
    args = (kc, vc, [0], [q.shape[0]], q, kn, vn, tau)
    ref, sigma = chunk_spread(*args)
    check_spread(gear.chunk_attn(*args, out_dtype=F32), ref, sigma, F32, what)
    assert gear.device_status() == 0


def groups(H, n, sizes, seed):
    """Values whose groups of 32 tokens have these deviations in turn."""
    s = torch.tensor(sizes, device="cuda")[torch.arange(n, device="cuda") // 32 % len(sizes)]
    return rnd(seed, H, n, 128, dt=F32) * s[None, :, None]


SIZES = [(0.0035, 0.0042), (0.004, 0.0035, 0.0036), (1e-4, 1.0), (1.0, 1e-4, 0.02), (300.0, 0.01)]


def peaked(dt, H, count, sizes, rank):
    """The first token takes half of the attention and has no value to speak of, 8192 others share the rest: their
    weights, 2^-13 of the first one's, are what the result is made of."""
    n = 8192
    top = rnd(1, 128, dt=F32)
    k, v = rnd(2, H, n, 128, dt=F32) * 0.1, groups(H, n, sizes, 3)
    k[:, 0], v[:, 0] = top, 0
    kc, vc = pair(n, dt, k, v, rank=rank, buffer_rank=0)
    q = (top * math.log(n) / TAU / top.square().sum() * (1 + 0.01 * rnd(4, count, 4 * H, 1, dt=F32))).to(dt)
    kn, vn = rnd(5, count, H, 128, dt=F32) * 0.1, rnd(6, count, H, 128, dt=F32) * sizes[-1]
    check(kc, vc, q, kn.to(dt), vn.to(dt), TAU, f"{dt} {sizes}")


@pytest.mark.parametrize("count", COUNTS)
@pytest.mark.parametrize("sizes", SIZES)
def test_values_of_mixed_size_under_a_peaked_softmax(count, sizes):
    for dt in [BF16] + [F16] * (max(sizes) < 2 and min(sizes) > 1e-3):
        peaked(dt, 16, count, sizes, 4)


@pytest.mark.parametrize("count", COUNTS)
@pytest.mark.parametrize("sizes", [(2.0 ** 40, 2.0 ** 38), (2.0 ** -40, 2.0 ** -42), (2.0 ** -12, 2.0 ** -14), (2.0 ** 16, 2.0 ** 13)])
def test_low_rank_values_far_from_one(count, sizes):
    """The low-rank part of bf16 values of any size: its factors stay in binary16's range."""
    peaked(BF16, 8, count, sizes, 4)
    n = 1500
    kc, vc = pair(n, BF16, rnd(1, 8, n, 128, dt=F32) * 0.3, groups(8, n, sizes, 3), bits=2, rank=8, buffer_rank=2)
    q, kn, vn = rnd(4, count, 32, 128, dt=BF16), rnd(5, count, 8, 128, dt=BF16), rnd(6, count, 8, 128, dt=F32) * sizes[0]
    check(kc, vc, q, kn, vn.to(BF16), TAU, "2 bits")


@pytest.mark.parametrize("count", COUNTS)
@pytest.mark.parametrize("rank", [4, 16])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_large_queries_and_low_rank_keys(dt, rank, count):
    """Queries of deviation 200 to 500, with a softmax scale as small: their products with the low-rank factors of
    prompts of 1024 tokens and more stay finite, and right."""
    for n, size, ks in ((1024, 200.0, 0.1), (1100, 500.0, 0.01), (1024, 900.0, 2.0), (6000, 900.0, 0.1), (1024, 0.002, 1.0)):
        k = rnd(1, 2, n, 128, dt=F32) * ks
        kc, vc = pair(n, dt, k, keys(2, 2, n, 128, dt=F32), rank=rank, buffer_rank=2)
        q = (rnd(3, count, 8, 128, dt=F32) * size).to(dt)
        kn, vn = rnd(4, count, 2, 128, dt=F32) * ks, rnd(5, count, 2, 128, dt=dt)
        check(kc, vc, q, kn.to(dt), vn, TAU / size / ks, f"{n} {size} {ks}")


@pytest.mark.parametrize("dt", [F16, BF16])
def test_queries_along_the_leading_direction(dt):
    """A query along a column of the low-rank factor, with a norm of 20 to 40000."""
    kc, vc = pair(2048, dt, rnd(1, 1, 2048, 128, dt=F32) * 0.05, keys(2, 1, 2048, 128, dt=F32), rank=4, buffer_rank=2)
    u = kc.arrays()["rfac"][0, 0, 0, :, 0].float()
    norms = torch.tensor([20.0, 400.0, 1500.0, 40000.0], device="cuda")
    for count in COUNTS:
        q = (u / u.norm() * norms[:, None]).expand(count, 4, 128).to(dt).contiguous()
        for size in norms.tolist():   # a scale that suits one of them: the others pick one token or weigh all alike
            got = gear.chunk_attn(kc, vc, [0], [count], q, None, None, 20 * TAU / size, out_dtype=F32)
            ref, bound = chunk_ref(kc, vc, [0], [count], q, None, None, 20 * TAU / size)
            check_chunk(got, ref, bound, F32, f"{count} {size}")
    assert gear.device_status() == 0


@pytest.mark.parametrize("count", COUNTS)
@pytest.mark.parametrize("codec", [dict(bits=2, group_size=32), dict(bits=4), dict(bits=8, group_size=128),
                                   dict(bits=4, meta_f16=True), dict(bits=4, kivi=True, buffer_len=64)])
def test_small_values_of_fp16_caches(codec, count):
    """Keys and values whose codes' scales lie near or below binary16's normal range lose no more than a rounding to it."""
    for ks, vs in ((1.0, 2e-4), (2e-4, 1.0), (1.0, 3e-5), (3e-3, 3e-3)):
        n = 700
        kc, vc = pair(n, F16, rnd(1, 2, n, 128, dt=F32) * ks, rnd(2, 2, n, 128, dt=F32) * vs, rank=4, buffer_rank=2, **codec)
        q = (rnd(3, count, 8, 128, dt=F32) / ks).to(F16)
        kn, vn = rnd(4, count, 2, 128, dt=F32) * ks, rnd(5, count, 2, 128, dt=F32) * vs
        check(kc, vc, q, kn.to(F16), vn.to(F16), TAU, f"{ks} {vs}")


@pytest.mark.parametrize("kivi", [False, True])
@pytest.mark.parametrize("bits", [2, 4, 8])
def test_values_up_to_the_end_of_fp16(bits, kivi):
    """Keys or values up to 65504, of which whole tokens lie there: compressed, buffered and the chunk's own."""
    codec = dict(bits=bits, kivi=kivi, buffer_len=64) if kivi else dict(bits=bits)
    for top in (20000.0, 60000.0, 65504.0):
        for big in ("keys", "values"):
            k, v = (((rnd(i, 2, 700, 128, dt=F32) / 3).clamp(-1, 1) * top if big == name else rnd(i, 2, 700, 128, dt=F32))
                    for i, name in ((1, "keys"), (2, "values")))
            k[:, 40], v[:, 50] = k[:, 40].sign() * k.abs().amax(), v[:, 50].sign() * v.abs().amax()
            kc, vc = pair(700, F16, k, v, rank=4, buffer_rank=2, **codec)
            new = [x[:, 30:60].transpose(0, 1).to(F16).contiguous() for x in (k, v)]
            gear.append_rope_rows(kc, vc, [0], [30], *new)
            for count in COUNTS:
                q = (rnd(3, count, 8, 128, dt=F32) / (top if big == "keys" else 1)).to(F16)
                kn, vn = (x[:, :count].transpose(0, 1).to(F16).contiguous() for x in (k, v))
                check(kc, vc, q, kn, vn, TAU, f"{top} {big} {count}")


@pytest.mark.parametrize("count", COUNTS)
def test_large_values_without_weight_beside_small_ones(count):
    """Every other 32 tokens have values 10000 times as large and next to no weight: the result is the small ones'."""
    n, H = 4096, 8
    top = rnd(1, 128, dt=F32)
    k, v = rnd(2, H, n, 128, dt=F32) * 0.1, groups(H, n, (1e-4, 1.0), 3)
    large = torch.arange(n, device="cuda") // 32 % 2 == 1
    k[:, large] = -4 * top
    k[:, 0], v[:, 0] = top, 0
    for dt in (BF16, F16):
        kc, vc = pair(n, dt, k, v, rank=0, buffer_rank=0)
        q = (top * math.log(n) / TAU / top.square().sum() * (1 + 0.01 * rnd(4, count, 4 * H, 1, dt=F32))).to(dt)
        check(kc, vc, q, None, None, TAU, f"{dt}")
