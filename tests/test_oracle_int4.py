"""The 4-bit cache's oracle and the host side of its calls, on the CPU: the
record's byte map against the header's words, quantisation against its
definition element by element, the argument checks of every call."""

import ctypes

import numpy as np
import pytest

from oracle import int4 as oi
from oracle import numerics as nx


def test_record_map_covers_every_byte_once():
    seen = np.zeros(oi.RECORD, dtype=int)
    for w in (0, 1):
        for t in range(64):
            for d in range(0, 128, 2):
                assert oi.byte_of(w, t, d) == oi.byte_of(w, t, d + 1)
                seen[oi.byte_of(w, t, d)] += 1
            for g in range(4):
                seen[oi.scale_byte(w, t, g)] += 1
                seen[oi.scale_byte(w, t, g) + 1] += 1
    assert np.all(seen == 1)


def test_quantise_is_the_nearest_code():
    r = np.random.default_rng(0)
    x = nx.bf16_round(r.standard_normal((50, 128)) * np.exp(r.standard_normal((50, 1)) * 4))
    c, s = oi.quantise(x)
    for i in range(50):
        for g in range(4):
            row, sc = x[i, 32 * g:32 * g + 32], s[i, g]
            assert sc == nx.bf16_round(np.abs(row).max() / 7)
            for e, code in zip(row, c[i, 32 * g:32 * g + 32]):
                err = [abs(e - k * sc) for k in range(-7, 8)]
                assert abs(e - code * sc) == min(err)
    assert np.abs(c).max() == 7


def test_quantise_special_groups():
    x = np.zeros((4, 128))
    x[1, 5] = np.nan
    x[2, 40] = -np.inf
    x[3] = 2.0 ** -140      # a / 7 is below half of bf16's smallest value
    c, s = oi.quantise(x)
    assert np.all(c == 0) and np.all(s[0] == 0) and np.all(s[3] == 0)
    assert np.isnan(s[1, 0]) and np.all(s[1, 1:] == 0)
    assert np.isnan(s[2, 1]) and s[2, 0] == 0


def test_write_and_read_rows_round_trip():
    r = np.random.default_rng(1)
    cache = np.full((3, 8, oi.RECORD), 0xFF, dtype=np.uint8)
    rows = {}
    for slot in r.permutation(192)[:100]:
        for h in (0, 7):
            k, v = nx.bf16_round(r.standard_normal((2, 128)))
            oi.write_row(cache, slot, h, k, v)
            rows[slot, h] = (k, v)
    for (slot, h), (k, v) in rows.items():
        K, V = oi.read_rows(cache, [slot // 64], h)
        assert np.array_equal(K[slot % 64], oi.values(k)) and np.array_equal(V[slot % 64], oi.values(v))


# ------------------------------------------------------- refusals (no kernel runs)

@pytest.fixture(scope="module")
def lib():
    from paged_gqa_decode_rope_gb300.build import build_library
    build_library()
    from paged_gqa_decode_rope_gb300 import _lib
    return _lib.lib()


P = ctypes.c_void_p(4096)      # never dereferenced on the host
ODD = ctypes.c_void_p(4098)
BAD, UNSUP = -1, -2


def test_refusals_of_the_prologue(lib):
    a = [P] * 5 + [16, P, P, 1e-6, P, 2, 4, P, None, 0, 1.0, P, 1, P, None]
    for i, v, rc in ((0, None, BAD), (10, 3, UNSUP), (14, 1, UNSUP), (17, -1, BAD), (9, ODD, BAD)):
        b = list(a)
        b[i] = v
        assert lib.hpc_rope_norm_kvwrite_ex(*b) == rc, (i, v)


def test_refusals_of_the_attention(lib):
    from paged_gqa_decode_rope_gb300._lib import AttnOptions, Plan
    plan = Plan(4096, 4096, 4096, 4096, 4096, 4096, 100, 10)
    a = [P, P, 2, None, 4, P, 8, P, 1, ctypes.byref(AttnOptions(1, 0, 1.0, 0)), ctypes.byref(plan), P, P,
         P, 0.1, P, None]
    for i, v, rc in ((0, ODD, BAD), (1, ODD, BAD), (2, 3, UNSUP), (4, 0, BAD), (4, 1 << 21, UNSUP),
                     (14, -0.1, BAD), (14, float("nan"), BAD),
                     (9, ctypes.byref(AttnOptions(1, 1, 1.0, 0)), UNSUP),
                     (9, ctypes.byref(AttnOptions(5, 0, 1.0, 0)), BAD)):
        b = list(a)
        b[i] = v
        assert lib.hpc_decode_attn_merge_ex(*b) == rc, (i, v)


def test_refusals_of_the_prefill(lib):
    a = [P, 8, P, P, 2, None, 4, P, 8, P, 1, P, P, P, 0, 0.1, P, None]
    assert lib.hpc_prefill_attn(*a) == UNSUP               # staged form only
    s = a[:16] + [P, 4, P, P, None]
    for i, v, rc in ((16, None, BAD), (17, 0, BAD), (18, None, BAD), (16, ODD, BAD), (4, 3, UNSUP)):
        b = list(s)
        b[i] = v
        assert lib.hpc_prefill_attn_staged(*b) == rc, (i, v)


def test_refusals_of_the_gather(lib):
    a = [P, 2, None, 4, P, 8, P, P, 0, P, None]
    for i, v, rc in ((0, None, BAD), (0, ODD, BAD), (1, 3, UNSUP), (1, 1, BAD), (3, 0, BAD), (4, None, BAD),
                     (5, -1, BAD), (6, ODD, BAD), (7, None, BAD), (8, 3, UNSUP), (9, None, BAD)):
        b = list(a)
        b[i] = v
        assert lib.hpc_kv_gather(*b) == rc, (i, v)
    a[5] = 0
    assert lib.hpc_kv_gather(*a) == 0                       # nothing to launch


def test_refusals_of_the_tables(lib):
    Q = ctypes.c_void_p(8192)
    a = [P, P, 4, 100, P, P, P, 8, Q, P, P, P, 16, P, None]
    cases = [(i, None, BAD) for i in (0, 1, 4, 5, 6, 8, 9, 10, 11, 13)]
    cases += [(2, -1, BAD), (2, 8193, UNSUP), (3, 0, BAD), (3, 1 << 21, UNSUP), (7, 0, BAD), (7, 1 << 25, UNSUP),
              (12, -1, BAD), (8, P, BAD)]
    for i, v, rc in cases:
        b = list(a)
        b[i] = v
        assert lib.hpc_block_tables(*b) == rc, (i, v)
    a = [P, P, 4, P, 8, 100, P, P, P, None]
    cases = [(i, None, BAD) for i in (0, 1, 3, 6, 7, 8)]
    cases += [(2, -1, BAD), (2, 8193, UNSUP), (4, 0, BAD), (4, 1 << 25, UNSUP), (5, 0, BAD)]
    for i, v, rc in cases:
        b = list(a)
        b[i] = v
        assert lib.hpc_block_release(*b) == rc, (i, v)
    a[2] = 0
    assert lib.hpc_block_release(*a) == 0


def test_queue_count_checks(lib):
    n = ctypes.c_int32(0)
    assert lib.hpc_decode_num_ctas(3, ctypes.byref(n)) == UNSUP
    assert lib.hpc_decode_num_queues(2, 5, 0, ctypes.byref(n)) == BAD


def test_refusals_of_the_step(lib):
    """Checked before the first of its two launches."""
    from paged_gqa_decode_rope_gb300._lib import Plan
    plan = Plan(4096, 4096, 4096, 4096, 4096, 4096, 100, 10)
    a = [P, P, P, P, P, 16, P, P, 1e-6, P, 2, 4, P, None, P, 8, P, 1, None, ctypes.byref(plan), P, P, P, P, 0.1, P,
         None]
    for i, v, rc in ((0, ODD, BAD), (9, ODD, BAD), (10, 3, UNSUP), (22, ODD, BAD), (24, -1.0, BAD)):
        b = list(a)
        b[i] = v
        assert lib.hpc_decode_step(*b) == rc, (i, v)


def test_arrays_without_entries_may_be_null(lib):
    assert lib.hpc_kv_gather(P, 2, None, 4, None, 0, None, None, 0, P, None) == 0
    assert lib.hpc_block_release(None, None, 0, None, 8, 100, P, P, P, None) == 0
    assert lib.hpc_kv_gather(P, 2, None, 4, None, 1, P, P, 0, P, None) == BAD
    assert lib.hpc_block_tables(None, None, 0, 100, P, P, None, 8, None, P, None, None, 1, P, None) == BAD
    assert lib.hpc_block_tables(None, P, 1, 100, P, P, P, 8, P, P, None, None, 0, P, None) == BAD


def test_bound_of_one_rounding_tells_one_from_two():
    """The bound that the decode attention is held to: P times the scale rounded
    to bf16 once, from fp32 or from P as a sum of two bf16, keeps it; rounding P
    first and the product again does not."""
    import int4_util as iu
    b = iu.Int4Batch([2, 3] * 20, 7, device=None)
    r = np.random.default_rng(8)
    worst = {"once": 0.0, "sum": 0.0, "twice": 0.0}
    bf = nx.bf16_round
    for s, L in enumerate(b.lengths):
        for h in range(8):
            n = -(-int(L) // 64)
            K, V = b.rows(s, h)
            q = bf(r.standard_normal(128))
            want, size = iu.attention(q, K, V, int(L))
            x = K @ q / np.sqrt(128)
            p = np.exp(x - x.max())[:, None]
            rec = b.host[b.table[s, :n], h]
            bits = rec[:, oi._SCALE[1]].astype(np.uint16) | (rec[:, oi._SCALE[1] + 1].astype(np.uint16) << 8)
            sc = np.repeat(nx.bf16_from_bits(bits).reshape(-1, 4)[:L], 32, axis=-1)
            codes = np.rint(V / sc)
            hi = bf(p)
            w = {"once": bf(p * sc), "sum": bf(hi * sc + bf(bf(p - hi) * sc)), "twice": bf(hi * sc)}
            for k, x in w.items():
                err = np.abs((x * codes).sum(0) / p.sum() - want)
                worst[k] = max(worst[k], float((err / (iu.WEIGHT_ONCE * size + 1e-30)).max()))
    assert worst["once"] < 1 and worst["sum"] < 1 < worst["twice"], worst
