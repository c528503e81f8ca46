"""Grouped-query attention over whole prompts and over the paged cache, and
the cache's writer, on the GPU through the public binding, against plain
64-bit forms (bounds: see gqa_reference)."""
import math

import pytest
import torch

from gqa_reference import U, attend, check, e4m3_rows

dsa = pytest.importorskip("sparse_attention_logits_b200")

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------ prompt --

# (prompt lengths, rows before the first prompt, rows behind the last, heads, kv heads, dim, dtype)
PROMPTS = {
    "one_token": ([1], 0, 0, 4, 4, 128, "bf16"),
    "one_token_d64": ([1], 0, 0, 2, 1, 64, "bf16"),
    "tile_edges": ([127, 128, 129, 1, 64], 0, 0, 8, 2, 128, "bf16"),
    "tile_edges_d64": ([255, 256, 257, 63, 65], 0, 0, 4, 2, 64, "bf16"),
    "empty_prompts": ([0, 0, 5, 0, 130, 0], 0, 0, 4, 2, 128, "bf16"),
    "rows_around": ([33, 70, 200], 19, 45, 4, 2, 128, "bf16"),
    "odd_group_of_3": ([300, 141, 17], 0, 0, 6, 2, 128, "bf16"),
    "mha_odd_heads": ([300, 141, 17], 0, 3, 3, 3, 128, "bf16"),
    "mqa_one_kv_head": ([500, 20], 0, 0, 16, 1, 64, "bf16"),
    "group_of_5_d64": ([400, 90], 5, 0, 5, 1, 64, "bf16"),
    "one_long": ([2049], 0, 0, 4, 1, 128, "bf16"),
    "long_and_short": ([1500, 3, 900, 1, 1, 1], 0, 0, 4, 2, 64, "bf16"),
    "many_short": ([(7 * i) % 23 for i in range(150)], 0, 0, 2, 2, 128, "bf16"),
    # few heads and long prompts: a row's keys in parts
    "parts": ([1500], 3, 9, 4, 1, 128, "bf16"),
    "parts_odd_group": ([1400, 300], 0, 0, 3, 1, 128, "bf16"),
    "parts_edges": ([768, 769, 513, 0, 1537], 2, 0, 2, 1, 64, "bf16"),
    "parts_one_head": ([130, 2600], 0, 1, 1, 1, 64, "bf16"),
    "fp32": ([1, 63, 64, 65, 0, 300], 2, 3, 6, 2, 64, "fp32"),
    "fp32_d128": ([200, 31], 0, 0, 4, 4, 128, "fp32"),
    "fp32_some_tiles": ([31, 900, 400], 1, 0, 8, 4, 64, "fp32"),
    "fp32_some_tiles_d128": ([900, 64, 3], 0, 2, 8, 2, 128, "fp32"),
    "fp32_many_tiles": ([700, 33, 800, 600], 0, 0, 16, 4, 64, "fp32"),
    "fp32_many_tiles_d128": ([129, 900], 0, 0, 16, 16, 128, "fp32"),
    "fp32_many_prompts": ([(29 * i) % 140 for i in range(40)], 0, 0, 4, 1, 64, "fp32"),
}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _prompt_inputs(case, seed=3):
    lens, before, behind, H, Hkv, D, dt = PROMPTS[case]
    total = before + sum(lens) + behind
    g = _gen(seed)
    # views of one fused projection's rows
    qkv = _randn((total, H + 2 * Hkv, D), g, DT[dt])
    cu = [before]
    for n in lens:
        cu.append(cu[-1] + n)
    # rows outside the prompts hold NaN: none may reach a prompt
    qkv[:before] = NAN
    qkv[cu[-1]:] = NAN
    return qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], cu


def _prompt_check(out, lse, q, k, v, cu, scale, a, b):
    n = b - a
    mask = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    ref, ref_lse, A, d = attend(q[a:b].transpose(0, 1), k[a:b].transpose(0, 1), v[a:b].transpose(0, 1), scale, mask)
    check(out[a:b].transpose(0, 1), lse[a:b].transpose(0, 1), ref, ref_lse, A, d, n, U[out.dtype])


@pytest.mark.parametrize("case", list(PROMPTS))
def test_prompt_attention(cuda_device, case):
    q, k, v, cu = _prompt_inputs(case)
    T, H, D = q.shape
    scale = 1.0 / math.sqrt(D)
    out = torch.full((T, H, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    dsa.gqa_prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), scale, out=out, lse=lse)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    for a, b in zip(cu, cu[1:]):
        if b > a:
            _prompt_check(out, lse, q, k, v, cu, scale, a, b)
    # rows outside every prompt are left as they were
    for part in (slice(0, cu[0]), slice(cu[-1], T)):
        assert bool((out[part] == 7).all()) and bool((lse[part] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_large_and_peaked_scores(cuda_device, dtype):
    """Scores of a few hundred, falling and rising along the keys: the running maximum moves all the time."""
    g = _gen(5)
    n, D = 700, 128
    q, k, v = (_randn((n, 2, D), g, DT[dtype]) for _ in range(3))
    k *= torch.linspace(0.1, 6.0, n, device="cuda")[:, None, None].to(DT[dtype])
    q[::3] *= -3
    out, lse = dsa.gqa_prompt_attention(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), 0.3)
    _prompt_check(out, lse, q, k, v, [0, n], 0.3, 0, n)


@pytest.mark.parametrize("group", [1, 2])
def test_prompt_parts_of_peaked_scores(cuda_device, group):
    """Rows whose keys are taken in parts: maxima that rise and fall from part to part, a prompt
    beside rows of NaN, the caller's workspace full of NaN."""
    g = _gen(8)
    n, D, cu = 1700, 128, [70, 1770]
    q, k, v = (_randn((n + 80, h, D), g, torch.bfloat16) for h in (2 * group, 2, 2))
    k[70:1770] *= (3.2 + 3 * torch.sin(torch.arange(n, device="cuda") / 150))[:, None, None].to(torch.bfloat16)
    for x in (q, k, v):
        x[:70] = NAN
        x[1770:] = math.inf
    need = dsa.gqa_prompt_attention_workspace_size(n + 80, 1, 2 * group, D, torch.bfloat16)
    assert need > 0
    ws = torch.full((need // 4,), NAN, device="cuda")
    out, lse = dsa.gqa_prompt_attention(q, k, v, _i32(cu), 0.3, workspace=ws.view(torch.uint8))
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    _prompt_check(out, lse, q, k, v, cu, 0.3, *cu)
    again = dsa.gqa_prompt_attention(q, k, v, _i32(cu), 0.3)
    assert torch.equal(out[70:1770], again[0][70:1770]) and torch.equal(lse[70:1770], again[1][70:1770])


@pytest.mark.parametrize("dtype,D,H,Hkv", [("bf16", 128, 4, 2), ("bf16", 64, 3, 1), ("fp32", 64, 2, 2)])
def test_prompts_never_reach_one_another(cuda_device, dtype, D, H, Hkv):
    """Prompts between others full of NaN and infinities, ending inside a tile of keys."""
    g = _gen(7)
    lens = [70, 61, 200, 3, 129, 50]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    qkv = _randn((cu[-1], H + 2 * Hkv, D), g, DT[dtype])
    for i in (0, 2, 4):
        qkv[cu[i]:cu[i + 1]] = math.inf if i == 2 else NAN
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    out, lse = dsa.gqa_prompt_attention(q, k, v, _i32(cu), 0.1)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    for i in (1, 3, 5):
        _prompt_check(out, lse, q, k, v, cu, 0.1, cu[i], cu[i + 1])


def test_prompt_nan_queries_stay_in_their_rows(cuda_device):
    q, k, v = (_randn((300, 2, 128), _gen(8), torch.bfloat16) for _ in range(3))
    clean = dsa.gqa_prompt_attention(q, k, v, _i32([0, 300]), 0.1)
    q = q.clone()
    q[[5, 130, 299]] = NAN
    out, lse = dsa.gqa_prompt_attention(q, k, v, _i32([0, 300]), 0.1)
    rows = torch.ones(300, dtype=torch.bool, device="cuda")
    rows[[5, 130, 299]] = False
    assert torch.equal(out[rows], clean[0][rows]) and torch.equal(lse[rows], clean[1][rows])
    assert bool(torch.isnan(out[~rows]).all())


# An fp32 NaN as torch fills it in, and as GPU arithmetic makes it.
NAN_BITS = {"filled": 0x7FC00000, "computed": 0x7FFFFFFF, "negative": -1}


def _nan(which):
    return _i32([NAN_BITS[which]]).view(torch.float32)[0]


@pytest.mark.parametrize("which", list(NAN_BITS))
@pytest.mark.parametrize("D", [64, 128])
def test_fp32_prompt_nan_queries_show_and_stay_in_their_rows(cuda_device, D, which):
    q, k, v = (_randn((300, 2, D), _gen(8)) for _ in range(3))
    clean = dsa.gqa_prompt_attention(q, k, v, _i32([0, 300]), 0.1)
    bad = [5, 130, 299]
    q = q.clone()
    q[bad, :, 7] = _nan(which)                              # one element of a row is enough
    out, lse = dsa.gqa_prompt_attention(q, k, v, _i32([0, 300]), 0.1)
    rows = torch.ones(300, dtype=torch.bool, device="cuda")
    rows[bad] = False
    assert torch.equal(out[rows], clean[0][rows]) and torch.equal(lse[rows], clean[1][rows])
    assert bool(torch.isnan(out[~rows]).all()) and bool(torch.isnan(lse[~rows]).all())


def test_fp32_prompt_largest_numbers(cuda_device):
    """Keys and values next to the largest fp32 number: their parts must not round up to infinity."""
    top, near = torch.finfo(torch.float32).max, float.fromhex("0x1.FFEp127")
    g, n = _gen(9), 40
    q, k, v = (_randn((n, 2, 64), g) for _ in range(3))
    q[:, :, 3] = 0
    k[:, 0, 3], k[:, 1, 3] = top, -top
    v[0, 0, 5], v[0, 1, 6] = near, -near                      # row 0 sees itself alone
    out, lse = dsa.gqa_prompt_attention(q, k, v, _i32([0, 1, n]), 0.1)
    for a, b in ((0, 1), (1, n)):
        _prompt_check(out, lse, q, k, v, None, 0.1, a, b)


@pytest.mark.parametrize("H,Hkv,D,n,places", [
    (4, 2, 128, 200, [*range(34), 63, 100, 127, 128, 140, 199]), (3, 1, 64, 300, [0, 1, 12, 13, 22, 23, 250, 258]),
    (1, 1, 64, 1800, [0, 13, 900, 1300])])                  # (the last: a row's keys in parts)
def test_prompt_nan_and_infinite_scores_show_at_any_place(cuda_device, H, Hkv, D, n, places):
    """A key that gives some row a NaN or an infinite score leaves NaN in that row, whichever key it is."""
    q, k, v = (_randn((n, h, D), _gen(10), torch.bfloat16) for h in (H, Hkv, Hkv))
    q[:, :, 5] = q[:, :, 5].abs() + 0.5
    clean = dsa.gqa_prompt_attention(q, k, v, _i32([0, n]), 0.1)
    for at in places:
        for bad in (NAN, math.inf):
            x = k.clone()
            x[at, :, 5] = bad
            out, lse = dsa.gqa_prompt_attention(q, x, v, _i32([0, n]), 0.1)
            assert bool(torch.isnan(out[at:]).all()) and bool(torch.isnan(lse[at:]).all()), (at, bad)
            assert torch.equal(out[:at], clean[0][:at]) and torch.equal(lse[:at], clean[1][:at]), (at, bad)


def test_prompt_row_strides_past_32_bits(cuda_device):
    """Rows 2.5 MB apart: the last lie more than 2^31 elements behind the first."""
    n, wide = 1800, 1250000
    big = torch.empty((n, wide), dtype=torch.bfloat16, device="cuda")
    part = _randn((n, 4, 64), _gen(9), torch.bfloat16)
    big[:, wide - 256:] = part.reshape(n, 256)
    x = big[:, wide - 256:].view(n, 4, 64)
    out, lse = dsa.gqa_prompt_attention(x[:, :2], x[:, 2:3], x[:, 3:], _i32([0, n]), 0.2)
    _prompt_check(out, lse, part[:, :2], part[:, 2:3], part[:, 3:], None, 0.2, 0, n)


def test_two_streams_at_once(cuda_device):
    """Calls that overlap on two streams, each with its own buffers: the results of the calls alone."""
    runs = []
    for seed in (1, 2):
        g = _gen(80 + seed)
        qkv = _randn((2000, 8, 128), g, torch.bfloat16)
        c = Paged([3000, 1234, 5], 2, 128, 16, "bf16", 90 + seed)
        q = _randn((3, 6, 128), g, torch.bfloat16)
        cu, b, p = _i32([0, 700, 2000]), _i32([0, 1, 2]), _i32([2999, 1233, 4])

        def run(qkv=qkv, c=c, q=q, cu=cu, b=b, p=p):
            return (*dsa.gqa_prompt_attention(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], cu, 0.1),
                    *dsa.gqa_decode_attention(q, c.k, c.v, c.table, b, p, 0.1))
        runs.append((run, run(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for run, _, stream in runs:
            with torch.cuda.stream(stream):
                got.append(run())
        torch.cuda.synchronize()
        for (_, want, _), x in zip(runs, got):
            assert all(torch.equal(a, b) for a, b in zip(want, x))


def test_prompt_bad_bounds_are_reported_and_skipped(cuda_device):
    g = _gen(6)
    q, k, v = (_randn((200, 2, 128), g, torch.bfloat16) for _ in range(3))
    for bounds in ([0, 100, 60, 200], [0, 100, 300], [-5, 100]):
        out = torch.zeros_like(q)
        lse = torch.zeros(200, 2, device="cuda")
        dsa.gqa_prompt_attention(q, k, v, torch.tensor(bounds, dtype=torch.int32, device="cuda"), 0.1, out=out, lse=lse)
        with pytest.raises(dsa.DSAError) as e:
            dsa.get_device_error(cuda_device)
        assert e.value.status == dsa.DSA_ERR_INVALID_ARG
        if bounds[0] == 0:
            _prompt_check(out, lse, q, k, v, bounds, 0.1, 0, 100 if bounds[2] != 60 else 60)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


# ------------------------------------------------------------------ decode --

class Paged:
    """A paged cache with every place that no sequence uses set to NaN."""

    def __init__(self, lens, hkv, D, page, kind, seed, spare=3):
        g = _gen(seed)
        self.page, self.kind = page, kind
        per = [-(-n // page) for n in lens]
        pages = sum(per) + spare
        width = max(max(per), 1) + 1
        ids = torch.randperm(pages, generator=g, device="cuda").tolist()
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(per[b]):
                table[b, j] = ids.pop()
                used[table[b, j], :min(page, n - j * page)] = True
        self.table = table.cuda()
        used = used.cuda()[:, None, :, None].expand(pages, hkv, page, D)
        out = []
        for _ in range(2):
            x = _randn((pages, hkv, page, D), g)
            if kind == "fp8":
                codes, scale = e4m3_rows(x * (0.05 + 4 * torch.rand((pages, hkv, page, 1), generator=g, device="cuda")))
                codes.view(torch.uint8).masked_fill_(~used, 0x7F)
                scale.masked_fill_(~used[..., 0], NAN)
                out += [codes, scale, codes.double() * scale.double()[..., None]]
            else:
                x = x.to(DT[kind]).masked_fill_(~used, NAN)
                out += [x, None, x.double()]
        self.k, self.k_scale, self.k64, self.v, self.v_scale, self.v64 = out

    def rows64(self, which, b, n):
        x = which[self.table[b, :-(-n // self.page)].long()]          # [pages, hkv, page, D]
        return x.transpose(0, 1).flatten(1, 2)[:, :n]


# (sequence lengths, rows per sequence, heads, kv heads, dim, page, cache)
DECODES = {
    "one_key": ([1], 1, 4, 1, 128, 16, "bf16"),
    "lengths_at_the_tile": ([63, 64, 65, 127, 128, 129], 1, 8, 2, 128, 64, "bf16"),
    "page_of_1": ([5, 40, 77], 1, 4, 2, 64, 1, "bf16"),
    "page_of_7": ([5, 40, 300], 1, 6, 2, 128, 7, "bf16"),
    "page_of_256": ([255, 700, 3], 1, 4, 4, 64, 256, "bf16"),
    "mha": ([100, 3, 1000], 1, 3, 3, 128, 16, "bf16"),
    "group_16": ([900, 33], 1, 32, 2, 128, 32, "bf16"),
    "group_17": ([500, 65], 1, 17, 1, 64, 32, "bf16"),
    "group_40": ([600, 5], 1, 40, 1, 128, 32, "bf16"),
    "group_5_rows_3": ([37, 2, 200], 3, 10, 2, 64, 16, "bf16"),
    "one_long_row": ([20011], 1, 8, 1, 128, 64, "bf16"),
    "many_rows": ([1 + (37 * i) % 190 for i in range(300)], 1, 8, 2, 64, 16, "bf16"),
    "ragged": ([4000, 1, 17, 2500, 600], 1, 16, 4, 128, 64, "bf16"),
    "fp8": ([63, 64, 65, 1, 1000], 1, 8, 2, 128, 64, "fp8"),
    "fp8_d64_odd_pages": ([400, 7, 33], 2, 6, 2, 64, 11, "fp8"),
    "fp8_group_17": ([500, 65], 1, 17, 1, 128, 16, "fp8"),
    "fp8_group_12": ([3000, 65], 1, 24, 2, 64, 16, "fp8"),
    "fp8_long": ([9001, 12], 1, 16, 2, 128, 64, "fp8"),
    "fp32": ([63, 64, 65, 1, 1000], 1, 8, 2, 128, 64, "fp32"),
    "fp32_d64_odd_pages": ([400, 7, 33], 2, 15, 3, 64, 5, "fp32"),
    "fp32_group_9": ([500, 65], 1, 9, 1, 128, 16, "fp32"),
}
U_P = {"bf16": U[torch.bfloat16], "fp8": U[torch.float16] + 2.0 ** -20, "fp32": U[torch.float32]}


def _decode_check(c, q, out, lse, batch, pos, scale):
    for r, (b, p) in enumerate(zip(batch, pos)):
        if p < 0:
            assert bool((out[r] == 0).all()) and bool(torch.isneginf(lse[r]).all())
            continue
        n = p + 1
        ref, ref_lse, A, d = attend(q[r][:, None], c.rows64(c.k64, b, n), c.rows64(c.v64, b, n), scale,
                                    torch.ones(1, n, dtype=torch.bool, device="cuda"))
        check(out[r][:, None], lse[r][:, None], ref, ref_lse, A, d, n, U_P[c.kind])


def _decode_case(case, seed=11):
    lens, per, H, Hkv, D, page, kind = DECODES[case]
    c = Paged(lens, Hkv, D, page, kind, seed)
    batch = [b for b in range(len(lens)) for _ in range(per)]
    pos = [max(-1, n - per + i) for n in lens for i in range(per)]
    g = _gen(seed + 1)
    fused = _randn((len(pos), H + 3, D), g, torch.float32 if kind == "fp32" else torch.bfloat16)
    return c, fused[:, 1:H + 1], batch, pos, 1.0 / math.sqrt(D)


@pytest.mark.parametrize("case", list(DECODES))
def test_decode_attention(cuda_device, case):
    c, q, batch, pos, scale = _decode_case(case)
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32(pos), scale, c.k_scale, c.v_scale)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    _decode_check(c, q, out, lse, batch, pos, scale)
    # the same call again gives the same bits (blocks' order does not matter)
    again = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32(pos), scale, c.k_scale, c.v_scale)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_decode_empty_rows_and_shuffled_batch(cuda_device, kind):
    """Padding rows anywhere, rows in any order of the sequences, one sequence twice."""
    lens = [130, 5, 900, 64]
    c = Paged(lens, 2, 128, 16, kind, 21)
    batch, pos = [2, 0, 0, 3, 1, 2, 0], [899, -1, 129, 63, 4, 500, -1]
    q = _randn((7, 6, 128), _gen(22), torch.float32 if kind == "fp32" else torch.bfloat16)
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32(pos), 0.2, c.k_scale, c.v_scale)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    _decode_check(c, q, out, lse, batch, pos, 0.2)
    # all rows empty
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32([-1] * 7), 0.2, c.k_scale, c.v_scale)
    _decode_check(c, q, out, lse, batch, [-1] * 7, 0.2)


# several rows of a sequence beside each other share its reads:
# (sequence lengths, [(sequence, position), ...], heads, kv heads, dim, page)
SHARED = {
    "drafts_of_4": ([1000, 7, 129, 4000], [(b, n - 4 + i) for b, n in enumerate([1000, 7, 129, 4000]) for i in range(4)],
                    8, 2, 128, 64),
    "drafts_of_2_d64": ([300, 128, 129], [(b, n - 2 + i) for b, n in enumerate([300, 128, 129]) for i in range(2)], 16, 2, 64, 16),
    "drafts_of_6_group_5": ([700, 64], [(b, n - 6 + i) for b, n in enumerate([700, 64]) for i in range(6)], 10, 2, 64, 5),
    "mha_of_20": ([500], [(0, 480 + i) for i in range(20)], 3, 3, 128, 16),
    "falling": ([900], [(0, p) for p in (899, 640, 639, 12)], 4, 1, 128, 64),
    "far_apart": ([3000], [(0, p) for p in (200, 2999, 5, 2600)], 4, 1, 64, 32),
    "one_place": ([777], [(0, 700)] * 5, 6, 2, 128, 64),
    "whole_units": ([1024], [(0, p) for p in (127, 255, 127, 511)], 8, 2, 128, 64),
    "empty_ones": ([400, 50], [(0, 399), (0, -1), (0, 380), (1, -1), (1, -1), (1, 49)], 4, 1, 128, 16),
    "uneven": ([600, 90, 10, 300], [(0, 599), (1, 85), (1, 86), (1, 87), (1, 88), (1, 89), (2, 9), (3, 290), (3, 291), (0, 12)],
               8, 2, 64, 16),
    "long": ([30000], [(0, 29997 + i) for i in range(3)], 5, 1, 64, 64),
    "many": ([40 + 9 * i for i in range(70)], [(b, 39 + 9 * b - i) for b in range(70) for i in range(3)], 8, 2, 64, 16),
    "very_many": ([20 + 5 * i for i in range(140)], [(b, 19 + 5 * b - i) for b in range(140) for i in range(2)], 4, 2, 64, 16),
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("case", list(SHARED))
def test_decode_rows_that_share_a_sequence(cuda_device, case, kind):
    lens, rows, H, Hkv, D, page = SHARED[case]
    c = Paged(lens, Hkv, D, page, kind, 23)
    batch, pos = [b for b, _ in rows], [p for _, p in rows]
    q = _randn((len(rows), H, D), _gen(24), torch.float32 if kind == "fp32" else torch.bfloat16)
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32(pos), 0.15, c.k_scale, c.v_scale)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    _decode_check(c, q, out, lse, batch, pos, 0.15)
    again = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32(pos), 0.15, c.k_scale, c.v_scale)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("n", [3, 130, 700])
def test_decode_rows_never_see_later_tokens(cuda_device, kind, n):
    """Four rows of a sequence whose last two tokens are NaN, infinite or 1e30 times the others."""
    D = 64
    c = Paged([n + 4, 50], 2, D, 16, kind, 25)
    batch, pos = [0, 0, 0, 0, 1], [n, n + 1, n + 2, n + 3, 49]
    q = _randn((5, 8, D), _gen(26), torch.float32 if kind == "fp32" else torch.bfloat16)

    def put(x, at, value):
        x[int(c.table[0, at // 16]), :, at % 16] = value
    for bad in (NAN, math.inf, 1e30):
        for at in (n + 2, n + 3):
            for x in (c.k_scale, c.v_scale) if kind == "fp8" else (c.k, c.v):
                put(x, at, bad)
        out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32(pos), 0.15, c.k_scale, c.v_scale)
        assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
        keep = [0, 1, 4]
        _decode_check(c, q[keep], out[keep], lse[keep], [0, 0, 1], [n, n + 1, 49], 0.15)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_decode_bad_rows_that_share_a_sequence(cuda_device, kind):
    """Rows of sequences out of range beside each other, and a page out of range that only the later rows reach."""
    c = Paged([300, 100], 2, 64, 16, kind, 27)
    table = c.table.clone()
    table[0, 18] = 10 ** 6                                  # tokens 288 .. 299
    batch, pos = [0, 0, 0, 9, 9, 9, 1, 1, 1, -1, -1], [285, 287, 299, 1, 2, 3, 97, 98, 99, 5, 6]
    q = _randn((len(pos), 6, 64), _gen(28), torch.float32 if kind == "fp32" else torch.bfloat16)
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, table, _i32(batch), _i32(pos), 0.15, c.k_scale, c.v_scale)
    with pytest.raises(dsa.DSAError) as e:
        dsa.get_device_error(cuda_device)
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG
    _decode_check(c, q, out, lse, [max(b, 0) if b < 2 else 0 for b in batch],
                  [p if b in (0, 1) else -1 for b, p in zip(batch, [285, 287, 287, *pos[3:]])], 0.15)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


def test_captured_rows_and_prompts_change_between_replays(cuda_device):
    """One captured graph of a decode of several rows a sequence and of prompts in parts; the rows'
    sequences and lengths, and the prompts' bounds, are others at each replay."""
    c = Paged([700, 260, 90], 1, 64, 16, "bf16", 29)
    n = 1300
    q, x = _randn((8, 4, 64), _gen(30), torch.bfloat16), _randn((n, 6, 64), _gen(31), torch.bfloat16)
    batch, pos, cu = _i32([0] * 8), _i32([-1] * 8), _i32([0, n])
    pq, pk, pv = x[:, :4], x[:, 4:5], x[:, 5:]

    def step():
        return (dsa.gqa_decode_attention(q, c.k, c.v, c.table, batch, pos, 0.15),
                dsa.gqa_prompt_attention(pq, pk, pv, cu, 0.15))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        (out, lse), (pout, plse) = step()
    for b, p, first in (([0] * 4 + [1] * 4, [696, 697, 698, 699, 40, 41, 42, 43], 0),
                        ([2, 2, 0, 1, 1, 1, 1, 0], [89, -1, 650, 256, 257, 258, 259, 0], 511),
                        ([1, 0, 1, 0, 2, 2, 2, 2], [5, 6, 7, 8, 80, 85, 60, 89], 1290)):
        batch.copy_(_i32(b))
        pos.copy_(_i32(p))
        cu.copy_(_i32([first, n]))
        graph.replay()
        torch.cuda.synchronize()
        _decode_check(c, q, out, lse, b, p, 0.15)
        _prompt_check(pout, plse, pq, pk, pv, [first, n], 0.15, first, n)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_decode_large_scores(cuda_device, kind):
    """Scores of a few hundred that grow along the sequence: every slice moves the maximum."""
    c = Paged([3000], 1, 128, 64, kind, 31)
    q = 4 * _randn((1, 8, 128), _gen(32), torch.float32 if kind == "fp32" else torch.bfloat16)
    if kind == "fp8":
        c.k_scale *= torch.linspace(0.2, 3, c.k_scale.numel(), device="cuda").reshape(c.k_scale.shape)
        c.k64 = c.k.double() * c.k_scale.double()[..., None]
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32([0]), _i32([2999]), 1.0, c.k_scale, c.v_scale)
    _decode_check(c, q, out, lse, [0], [2999], 1.0)


@pytest.mark.parametrize("which", list(NAN_BITS))
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 64), (8, 2, 128), (24, 2, 64)])
def test_fp32_decode_nan_is_not_lost(cuda_device, H, Hkv, D, which):
    """A NaN in a query, or in a visible key or value, shows in everything that it takes part in, and there alone."""
    lens, g = [50, 777], H // Hkv
    c = Paged(lens, Hkv, D, 16, "fp32", 33)
    q = _randn((2, H, D), _gen(34))

    def run(q):
        return dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32([0, 1]), _i32([49, 776]), 0.15)
    clean = run(q)
    bad = q.clone()
    bad[1, 3, 7] = _nan(which)
    out, lse = run(bad)
    hit = torch.zeros(2, H, dtype=torch.bool, device="cuda")
    hit[1, 3] = True
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
    for b, at in ((0, 0), (0, 49), (1, 401)):
        hit = torch.zeros(2, H, dtype=torch.bool, device="cuda")
        hit[b, g:] = True                                   # (kv head 1)
        for cache in (c.k, c.v):
            place = cache[int(c.table[b, at // 16]), 1, at % 16]
            was = place[9].clone()
            place[9] = _nan(which)
            out, lse = run(q)
            place[9] = was
            assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
            if cache is c.k:
                assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
            else:
                dims = torch.arange(D, device="cuda") == 9
                assert bool(torch.isnan(out[hit][:, dims]).all()) and torch.equal(lse[hit], clean[1][hit])
                assert torch.equal(out[hit][:, ~dims], clean[0][hit][:, ~dims])


def test_fp32_decode_largest_numbers(cuda_device):
    """Keys and values next to the largest fp32 number: their parts must not round up to infinity."""
    top, near = torch.finfo(torch.float32).max, float.fromhex("0x1.FFEp127")
    c = Paged([1, 90], 2, 64, 16, "fp32", 35)
    q = _randn((2, 4, 64), _gen(36))
    q[:, :, 3] = 0
    for b, n in ((0, 1), (1, 90)):
        for at in range(n):
            c.k[int(c.table[b, at // 16]), :, at % 16, 3] = top if at % 2 else -top
    c.v[int(c.table[0, 0]), 0, 0, 5], c.v[int(c.table[0, 0]), 1, 0, 6] = near, -near      # (sequence 0 has one token)
    c.k64, c.v64 = c.k.double(), c.v.double()
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32([0, 1]), _i32([0, 89]), 0.15)
    _decode_check(c, q, out, lse, [0, 1], [0, 89], 0.15)


@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_decode_nan_shows_at_any_length(cuda_device, kind, group):
    """A row of a NaN query, and one whose first half of keys is NaN, are NaN whether a block holds the whole row or
    many blocks hold parts of it; the rows beside them stand."""
    lens = [50, 777, 20000, 20000, 300, 30]
    c = Paged(lens, 2, 64, 16, kind, 37)
    q = _randn((6, 2 * group, 64), _gen(38), torch.float32 if kind == "fp32" else torch.bfloat16)
    for r in (0, 1, 2):
        q[r, :, 11] = NAN
    (c.k_scale if kind == "fp8" else c.k)[c.table[3, :625].long()] = NAN
    pos = [n - 1 for n in lens]
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(range(6)), _i32(pos), 0.15, c.k_scale, c.v_scale)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    for r in range(4):
        assert bool(torch.isnan(out[r]).all()) and bool(torch.isnan(lse[r]).all()), r
    _decode_check(c, q[4:], out[4:], lse[4:], [4, 5], pos[4:], 0.15)


@pytest.mark.parametrize("H,Hkv,D,per", [(8, 2, 128, 1), (8, 2, 64, 1), (24, 2, 64, 1), (16, 1, 128, 1), (4, 2, 64, 3), (8, 2, 128, 2)])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4, 1e-6])
def test_decode_fp8_zero_rows_beside_small_values(cuda_device, size, H, Hkv, D, per):
    """All-zero value rows (codes +0 or -0) have the scale 1, however small the others' values are; beside them rows that
    are zero but for a few dims, and count."""
    lens = [9000, 200]
    c = Paged(lens, Hkv, D, 16, "fp8", 39)
    c.v_scale *= size
    zero = torch.arange(c.v.shape[0] * Hkv * 16, device="cuda").reshape(c.v.shape[:3]) % 13 == 4
    zero &= ~torch.isnan(c.v_scale)
    codes = c.v.view(torch.uint8)
    codes[zero] = torch.where(torch.arange(D, device="cuda") % 3 == 0, 0x80, 0).to(torch.uint8)
    c.v_scale[zero] = 1.0
    few = torch.arange(zero.numel(), device="cuda").reshape(zero.shape) % 13 == 9
    codes[..., :D - 5][few & ~torch.isnan(c.v_scale)] = 0
    c.v64 = c.v.double() * c.v_scale.double()[..., None]
    batch = [b for b in range(2) for _ in range(per)]
    pos = [n - per + i for n in lens for i in range(per)]
    q = _randn((2 * per, H, D), _gen(40), torch.bfloat16)
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32(batch), _i32(pos), 0.15, c.k_scale, c.v_scale)
    _decode_check(c, q, out, lse, batch, pos, 0.15)


@pytest.mark.parametrize("group", [1, 9])
@pytest.mark.parametrize("ratio", [1e3, 1e8])
def test_decode_fp8_value_scales_far_apart(cuda_device, ratio, group):
    """A token of next to no weight whose value scale is far above the others', one token that holds most of the weight,
    and thousands that share the rest.  300 rows over the same pages, so that a block meets a row's keys one after another."""
    n, D, rows = 5000, 128, 300
    c = Paged([n], 1, D, 16, "fp8", 41)
    q1 = _randn((D,), _gen(42), torch.bfloat16)
    q = q1.expand(rows, group, D).contiguous()
    scale, unit = 0.1, q1.float() / float((q1.float() ** 2).sum())

    def put(at, z, v_scale):                                # a key of score z; its value's scale
        page, slot = int(c.table[0, at // 16]), at % 16
        codes, s = e4m3_rows((unit * (z / scale))[None])
        c.k.view(torch.uint8)[page, 0, slot], c.k_scale[page, 0, slot] = codes.view(torch.uint8)[0], s[0]
        c.v_scale[page, 0, slot] *= v_scale
    c.k_scale *= 1e-3                                       # scores of nearly 0
    put(3, 11.5, 1e-3)
    put(17, -2.0 * math.log(ratio), ratio)
    put(3333, -60.0, ratio)
    c.k64, c.v64 = (x.double() * s.double()[..., None] for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    table = c.table.expand(rows, -1).contiguous()
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, table, _i32(range(rows)), _i32([n - 1] * rows), scale, c.k_scale, c.v_scale)
    for r in (0, 1, 2, 137, rows - 1):
        _decode_check(c, q[r:r + 1], out[r:r + 1], lse[r:r + 1], [0], [n - 1], scale)


@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("scale", [1e-7, 1e-9, 1e-30])
def test_decode_fp8_zero_query_and_small_scale(cuda_device, scale, group):
    """Queries of zeros (padding) see the mean of the values at any scale."""
    c = Paged([45, 300], 1, 64, 16, "fp8", 43)
    q = torch.zeros((2, group, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = dsa.gqa_decode_attention(q, c.k, c.v, c.table, _i32([0, 1]), _i32([44, 299]), scale, c.k_scale, c.v_scale)
    _decode_check(c, q, out, lse, [0, 1], [44, 299], scale)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_decode_bad_indexes_are_reported(cuda_device, kind):
    lens = [200, 100]
    c = Paged(lens, 2, 64, 16, kind, 41)
    q = _randn((3, 4, 64), _gen(42), torch.float32 if kind == "fp32" else torch.bfloat16)

    def run(batch, pos, table=c.table):
        out, lse = dsa.gqa_decode_attention(q, c.k, c.v, table, _i32(batch), _i32(pos), 0.1, c.k_scale, c.v_scale)
        with pytest.raises(dsa.DSAError) as e:
            dsa.get_device_error(cuda_device)
        assert e.value.status == dsa.DSA_ERR_INVALID_ARG
        return out, lse
    # a sequence out of range: as an empty row; the others stand
    out, lse = run([0, 7, 1], [199, 5, 99])
    _decode_check(c, q, out, lse, [0, 0, 1], [199, -1, 99], 0.1)
    out, lse = run([0, -1, 1], [199, 5, 99])
    _decode_check(c, q, out, lse, [0, 0, 1], [199, -1, 99], 0.1)
    # a position past the table's width, and a page out of range: left out
    for table, batch, pos in ((c.table, [0, 1, 1], [199, 10 ** 6, 99]), (c.table.clone(), [0, 1, 1], [199, 50, 99])):
        if pos[1] == 50:
            table[0, 3] = 10 ** 6
        out, lse = run(batch, pos, table)
        assert bool(torch.isfinite(lse[::2]).all())         # (row 1 of the first names places that hold NaN)
        _decode_check(c, q[2:], out[2:], lse[2:], [1], [99], 0.1)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


def test_cache_offsets_past_32_bits(cuda_device):
    """Pages whose first elements lie beyond 2^31 elements (and 2^32 bytes) of the cache: written, read and copied."""
    pages, hkv, page, D = 17000, 8, 128, 128                # 2.2e9 elements, 4.5 GB a cache
    k_cache, v_cache = (torch.empty((pages, hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = _i32([[pages - 1, 3, pages - 2], [pages - 3, pages - 4, 5]])
    n = 300
    g = _gen(43)
    batch = torch.arange(2, device="cuda", dtype=torch.int32).repeat_interleave(n)
    pos = torch.arange(n, device="cuda", dtype=torch.int32).repeat(2)
    k, v = (_randn((2 * n, hkv, D), g, torch.bfloat16) for _ in "kv")
    dsa.kv_cache_append(k, v, batch, pos, table, k_cache, v_cache)
    q = _randn((2, 16, D), g, torch.bfloat16)

    def check_rows(t):
        out, lse = dsa.gqa_decode_attention(q, k_cache, v_cache, t, _i32([0, 1]), _i32([n - 1, n - 1]), 0.1)
        for r in range(2):
            part = slice(r * n, (r + 1) * n)
            ref, ref_lse, A, d = attend(q[r][:, None], k[part].transpose(0, 1), v[part].transpose(0, 1), 0.1,
                                        torch.ones(1, n, dtype=torch.bool, device="cuda"))
            check(out[r][:, None], lse[r][:, None], ref, ref_lse, A, d, n, U[torch.bfloat16])
    check_rows(table)
    dsa.kv_pages_copy([k_cache, v_cache], _i32([pages - 1, 3]), _i32([7, pages - 6]))
    check_rows(_i32([[7, pages - 6, pages - 2], [pages - 3, pages - 4, 5]]))
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


def test_decode_side_stream_and_caller_buffers(cuda_device):
    c, q, batch, pos, scale = _decode_case("ragged")
    b, p = _i32(batch), _i32(pos)
    ref = dsa.gqa_decode_attention(q, c.k, c.v, c.table, b, p, scale)
    need = dsa.gqa_decode_attention_workspace_size(q.shape[0], q.shape[1], c.k.shape[1], q.shape[2], c.k.dtype)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN everywhere: nothing of it is read first
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dsa.gqa_decode_attention(q, c.k, c.v, c.table, b, p, scale, out=out, lse=lse, workspace=ws)
    s.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_captured_decode_follows_growing_lengths(cuda_device):
    """One captured step (append, then attention) replayed while its position and input buffers change; a second
    graph that shares the workspace runs in between."""
    c = Paged([400, 400], 2, 128, 16, "bf16", 51)
    c.k[:] = _randn(c.k.shape, _gen(52), torch.bfloat16)
    c.v[:] = _randn(c.v.shape, _gen(53), torch.bfloat16)
    g = _gen(54)
    b, p = _i32([0, 1]), _i32([10, 10])
    qkv = _randn((2, 8 + 4, 128), g, torch.bfloat16)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    need = dsa.gqa_decode_attention_workspace_size(2, 8, 2, 128, torch.bfloat16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, device="cuda")) for _ in "ab"]

    def step(o):
        dsa.kv_cache_append(k, v, b, p, c.table, c.k, c.v)
        dsa.gqa_decode_attention(q, c.k, c.v, c.table, b, p, 0.1, out=o[0], lse=o[1], workspace=ws)
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(outs[0])
    torch.cuda.current_stream().wait_stream(side)
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(o)
        graphs.append(graph)
    for i, at in enumerate((11, 250, 12, 399, 64)):
        p.copy_(_i32([at, max(0, at - 5)]))
        qkv.copy_(_randn(qkv.shape, g, torch.bfloat16))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        c.k64, c.v64 = c.k.double(), c.v.double()
        pos = p.tolist()
        for r in range(2):
            assert torch.equal(c.rows64(c.k64, r, pos[r] + 1)[:, -1], k[r].double())
        _decode_check(c, q, *outs[i % 2], [0, 1], pos, 0.1)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("kind,src,D,page,hkv", [
    ("bf16", "bf16", 128, 64, 8), ("bf16", "fp32", 64, 16, 3), ("fp32", "fp32", 128, 7, 2), ("fp32", "fp32", 64, 1, 1),
    ("fp8", "bf16", 128, 64, 4), ("fp8", "fp32", 64, 5, 3), ("fp8", "bf16", 64, 16, 1)])
@pytest.mark.parametrize("n", [1, 2, 67, 1500])
def test_append(cuda_device, kind, src, D, page, hkv, n):
    """Rows land whole in their places, rounded once by the cache's rule, and nothing else changes."""
    g = _gen(61)
    B, width = 5, -(-400 // page)
    pages = B * width + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:B * width].reshape(B, width).to(torch.int32)
    where = torch.randperm(B * 400, generator=g, device="cuda")[:n]
    batch, pos = (where // 400).to(torch.int32), (where % 400).to(torch.int32)
    if n > 2:
        pos[1] = -1                                                    # not stored
    x = _randn((n, 2 + 2 * hkv, D), g, DT[src])
    if n > 2:
        x[2] = 0                                                       # all-zero rows: scale 1
        x[3] *= 1e-3
        x[4, :, 5] = 300
    k, v = x[:, 1:1 + hkv], x[:, 1 + hkv:1 + 2 * hkv]
    dt = {"fp8": torch.float8_e4m3fn, **DT}[kind]
    before = [torch.randint(0, 120, (pages, hkv, page, D * dt.itemsize), generator=g, device="cuda").to(torch.uint8).view(dt)
              for _ in "kv"]
    scales = [torch.rand((pages, hkv, page), generator=g, device="cuda") for _ in "kv"] if kind == "fp8" else [None, None]
    caches, sc = [t.clone() for t in before], [None if t is None else t.clone() for t in scales]
    dsa.kv_cache_append(k, v, batch, pos, table, caches[0], caches[1], sc[0], sc[1])
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    keep = pos >= 0
    pg = table[batch[keep].long(), (pos[keep] // page).long()].long()
    sl = (pos[keep] % page).long()
    for new, old, s_new, s_old, rows in zip(caches, before, sc, scales, (k, v)):
        rows = rows[keep]
        if kind == "fp8":
            codes, s = e4m3_rows(rows.float())
            s_old[pg, :, sl] = s
            assert torch.equal(s_new, s_old)
            old.view(torch.uint8)[pg, :, sl] = codes.view(torch.uint8)
        else:
            old[pg, :, sl] = rows.to(dt)
        assert torch.equal(new.view(torch.uint8), old.view(torch.uint8))


def test_append_bad_indexes_are_reported_and_skipped(cuda_device):
    k_cache = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    table = _i32([[0, 1], [9, -1]])
    x = torch.ones(5, 1, 64, dtype=torch.bfloat16, device="cuda")
    # good; page out of range; no page; past the table; no such sequence
    dsa.kv_cache_append(x, x, _i32([0, 1, 1, 0, 2]), _i32([17, 3, 20, 32, 0]), table, k_cache, v_cache)
    with pytest.raises(dsa.DSAError):
        dsa.get_device_error(cuda_device)
    assert bool((k_cache[1, 0, 1] == 1).all()) and float(k_cache.sum()) == 64 and float(v_cache.sum()) == 64


# ---------------------------------------------------------------- together --

@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_prompt_then_decode_over_the_cache(cuda_device, kind):
    """A serving run: room for two prompts, their keys and values stored, the prompts' attention; then one token at a
    time.  The cache's attention at the prompts' rows agrees with the prompts' own, and each new token with the
    64-bit form over all tokens so far; a branch and its parent go on apart; drawing the pool together changes nothing."""
    dt, D, H, Hkv, page, g = DT[kind], 64, 6, 2, 16, _gen(71)
    lens, B, width, pages = [37, 90], 3, 10, 40
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    length, count = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    k_cache = torch.full((pages, Hkv, page, D), NAN, dtype=dt, device="cuda")
    v_cache = torch.full_like(k_cache, NAN)
    u, scale = U[dt], 0.2
    count[:5] = 1                                                       # pages held by someone else
    dsa.kv_pages_extend(table, length, count, _i32([0, 2]), _i32(lens), page)
    total = sum(lens)
    qkv = _randn((total, H + 2 * Hkv, D), g, dt)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    batch = _i32([0] * lens[0] + [2] * lens[1])
    pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in lens])
    dsa.kv_cache_append(k, v, batch, pos, table, k_cache, v_cache)
    out, lse = dsa.gqa_prompt_attention(q, k, v, _i32([0, lens[0], total]), scale)
    out2, lse2 = dsa.gqa_decode_attention(q, k_cache, v_cache, table, batch, pos, scale)
    for a, b in ((0, lens[0]), (lens[0], total)):
        _prompt_check(out, lse, q, k, v, None, scale, a, b)
        _prompt_check(out2, lse2, q, k, v, None, scale, a, b)
    # sequence 1 branches off sequence 2; then all three take new tokens
    dsa.kv_pages_fork(table, length, count, _i32([2]), _i32([1]), page, [k_cache, v_cache])
    story = {0: (k[:lens[0]], v[:lens[0]]), 1: (k[lens[0]:], v[lens[0]:]), 2: (k[lens[0]:], v[lens[0]:])}
    rows = _i32([0, 1, 2])
    for step in range(20):
        if step == 10:
            dsa.kv_pages_compact(table, count, [k_cache, v_cache], table_out=table, ref_out=count)
            assert int((count > 0).sum()) == int((count[:int((count > 0).sum())] > 0).sum())
        dsa.kv_pages_extend(table, length, count, rows, _i32([1, 1, 1]), page)
        new = _randn((3, H + 2 * Hkv, D), g, dt)
        dsa.kv_cache_append(new[:, H:H + Hkv], new[:, H + Hkv:], rows, length - 1, table, k_cache, v_cache)
        o, l = dsa.gqa_decode_attention(new[:, :H], k_cache, v_cache, table, rows, length - 1, scale)
        for b in range(3):
            story[b] = (torch.cat([story[b][0], new[b:b + 1, H:H + Hkv]]), torch.cat([story[b][1], new[b:b + 1, H + Hkv:]]))
            n = story[b][0].shape[0]
            ref, ref_lse, A, d = attend(new[b, :H][:, None], story[b][0].transpose(0, 1), story[b][1].transpose(0, 1), scale,
                                        torch.ones(1, n, dtype=torch.bool, device="cuda"))
            check(o[b][:, None], l[b][:, None], ref, ref_lse, A, d, n, u)
    assert dsa.get_device_error(cuda_device) == dsa.DSA_OK
    assert length.tolist() == [57, 110, 110]


def test_calls_without_rows(cuda_device):
    """Empty batches: nothing is launched, outputs are empty, what the caches hold stays."""
    kc, vc = (torch.ones((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table, none = _i32([[0, 1]]), _i32([])
    x = torch.empty((0, 6, 64), dtype=torch.bfloat16, device="cuda")
    before = dsa.launch_count()
    dsa.kv_cache_append(x[:, :2], x[:, 2:4], none, none, table, kc, vc)
    for out, lse in (dsa.gqa_decode_attention(x, kc, vc, table, none, none, 0.1),
                     dsa.gqa_prompt_attention(x, x[:, :2], x[:, :2], _i32([0, 0]), 0.1)):
        assert out.shape == (0, 6, 64) and lse.shape == (0, 6)
    y = torch.ones((3, 6, 64), dtype=torch.bfloat16, device="cuda")
    kept = torch.full_like(y, 7.0)
    dsa.gqa_prompt_attention(y, y[:, :2], y[:, :2], _i32([0]), 0.1, out=kept)
    assert bool((kept == 7).all()) and bool((kc == 1).all()) and bool((vc == 1).all())
    assert dsa.launch_count() == before


@pytest.mark.parametrize("D", [64, 128])
def test_fp8_caches_as_bytes(cuda_device, D):
    """A uint8 cache holds the codes of a float8 one: written and read alike."""
    g, n = _gen(73), 90
    table = _i32([[3, 0, 5, 1, 2, 4]])
    k, v = (_randn((n, 2, D), g, torch.bfloat16) for _ in "kv")
    batch, pos, q = _i32([0] * n), torch.arange(n, device="cuda", dtype=torch.int32), _randn((1, 8, D), g, torch.bfloat16)
    got = []
    for dt in (torch.float8_e4m3fn, torch.uint8):
        caches = [torch.zeros((6, 2, 16, D), dtype=torch.uint8, device="cuda").view(dt) for _ in "kv"]
        scales = [torch.zeros((6, 2, 16), device="cuda") for _ in "kv"]
        dsa.kv_cache_append(k, v, batch, pos, table, *caches, *scales)
        got.append([x.view(torch.uint8) for x in caches] + scales +
                   list(dsa.gqa_decode_attention(q, *caches, table, _i32([0]), _i32([n - 1]), 0.1, *scales)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
