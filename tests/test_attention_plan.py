"""How attention is cut along the cache (host code, no GPU needed): the parts that the thread blocks count from a sequence's
length never exceed the parts that the launch and the workspace were made for."""
import ctypes
import itertools
import random

import pytest

from block_quantized_int8_q8_gb300 import _build, api


class Plan(ctypes.Structure):                                 # AttnPlan of csrc/attn.h
    _fields_ = [("few", ctypes.c_bool), ("chunk", ctypes.c_int), ("splits", ctypes.c_int), ("window", ctypes.c_int),
                ("part_o", ctypes.c_size_t), ("part_ml", ctypes.c_size_t), ("total", ctypes.c_size_t)]

    def same(self, other):
        return all(getattr(self, f) == getattr(other, f) for f, _ in self._fields_)


@pytest.fixture(scope="module")
def plan():
    _build.build()
    f = getattr(api.load(), "_ZN3mmq14attention_planExiiiixxx")
    f.argtypes = [ctypes.c_int64] + [ctypes.c_int] * 4 + [ctypes.c_int64] * 3
    f.restype = Plan
    return f


def device_parts(length, n, chunk, causal, window, max_tokens, max_kv):
    """visible_range of csrc/attn_math.cuh."""
    first, end = length - n, min(length, max_kv)
    j0 = max(first - window + 1, 0) if window > 0 else 0
    j1 = min(end, first + min(n, max_tokens)) if causal else end
    tiles = max((j1 + 15) // 16 - j0 // 16, 0)
    return max(-(-tiles * 16 // chunk), 1)


SIZES = [(8, 32, 8, 128, 8, 1, 8192), (1, 8, 2, 64, 1, 1, 131072), (4 * 2048, 32, 8, 128, 4, 2048, 4096),
         (2048, 16, 2, 256, 1, 2048, 32768), (3, 3, 1, 64, 2, 2, 1), (64, 64, 8, 128, 64, 1, (1 << 31) - 5000)]


@pytest.mark.parametrize("tokens,heads,kv,dim,seqs,most,max_kv", SIZES)
def test_windows_that_hide_nothing_are_no_window(plan, tokens, heads, kv, dim, seqs, most, max_kv):
    whole = plan(tokens, heads, kv, dim, seqs, most, max_kv, 0)
    assert whole.window == 0
    for window in (max_kv, max_kv + 1, max_kv + most, max_kv + most + 1, 1 << 31, (1 << 31) + 5, 1 << 32, 1 << 62,
                   (1 << 63) - 40, (1 << 63) - 1):
        assert plan(tokens, heads, kv, dim, seqs, most, max_kv, window).same(whole), window


def test_parts_fit_the_launch_and_the_workspace(plan):
    rng = random.Random(3)
    for _ in range(4000):
        kv, dim = rng.choice([1, 2, 8]), rng.choice([64, 128, 256])
        heads, seqs = kv * rng.choice([1, 3, 4, 8, 16]), int(2 ** rng.uniform(0, 9))
        most, max_kv = int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 18))
        tokens = rng.randint(max(most, seqs), seqs * most) if seqs * most > max(most, seqs) else max(most, seqs)
        window = rng.choice([0, 0, 1, 16, 100, max_kv // 2, max_kv, max_kv + most, 1 << 62, (1 << 63) - 1,
                             int(2 ** rng.uniform(0, 18))])
        p, whole = (plan(tokens, heads, kv, dim, seqs, most, max_kv, w) for w in (window, 0))
        assert p.total <= whole.total and p.chunk > 0 and p.chunk % 16 == 0
        # a sum of the tensor cores runs over 32768 tokens at most: longer parts put it aside in the workspace
        assert p.chunk <= 2048 if p.few else (p.total > 0) == (p.splits > 1 or p.chunk > 32768)
        assert p.total > 0 or p.splits == 1
        if p.total > 0:
            rows = tokens * heads * p.splits
            assert p.part_o >= rows * 8 and p.total - p.part_o >= rows * dim * 4
        for length, n, causal in itertools.product({0, 1, max_kv - 1, max_kv, max_kv + 7, rng.randint(0, max_kv)},
                                                   {1, most, most + 3, rng.randint(1, most)}, (True, False)):
            if causal or p.window == 0:
                assert device_parts(max(length, 0), n, p.chunk, causal, p.window, most, max_kv) <= p.splits
