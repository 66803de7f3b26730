"""Stream order between the library's own kernels, which all are launched with
programmatic stream serialization: each may start while the one before it
drains. The rules that order rests on are read from the sources (no GPU), and
the chains that depend on them are run."""
import glob
import os
import re

import numpy as np
import pytest

import token_sampling_logits_gb300 as gs
from token_sampling_logits_gb300 import build

gpu = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---- the sources ----------------------------------------------------------------
def _without_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", " ", text, flags=re.S)


def kernels():
    """(name, body) of every kernel but the diagnostic ones, which are launched
    without the attribute."""
    found = {}
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu"))):
        text = _without_comments(open(path).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\(", text):
            start = text.index("{", m.end())
            depth, i = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            found[m.group(1)] = text[start:i]
    return {k: v for k, v in found.items() if not k.startswith(("debug_", "probe_"))}


WAIT = re.compile(r"pdl_wait\w*\(\)|griddepcontrol\.wait")


def test_the_kernels_are_found():
    assert {"sample_kernel", "list_kernel", "sample_cluster_kernel", "hlg_kernel",
            "categorical_kernel", "filter_cluster_kernel", "process_kernel",
            "process_wide_kernel", "history_append_kernel", "history_append_long_kernel",
            "bias_set_kernel", "state_reset_kernel"} <= set(kernels())


@pytest.mark.parametrize("name", sorted(kernels()))
def test_every_kernel_waits_before_it_may_exit(name):
    """A kernel whose blocks all exit without having waited ends before its
    predecessor does, and its successor's wait covers it alone."""
    body = kernels()[name]
    wait, leave = WAIT.search(body), re.search(r"\breturn\b", body)
    assert wait, name
    assert leave is None or wait.start() < leave.start(), name


@pytest.mark.parametrize("name", ["process_kernel", "process_wide_kernel"])
def test_kernels_that_write_logits_do_not_release_early(name):
    """The samplers read logits through non-coherent loads, which may not read
    what is written during their kernel's life."""
    assert not re.search(r"release|launch_dependents", kernels()[name])


@pytest.mark.parametrize("name", ["bias_set_kernel", "history_append_kernel",
                                  "history_append_long_kernel"])
def test_lists_are_read_past_l1(name):
    """A list may be what a sampler, or a kernel that writes logits, just wrote."""
    text = _without_comments(open(os.path.join(build.CSRC, "gsample_constrain.cu")).read())
    body = kernels()[name]
    body += text[text.index("token_place("):text.index("history_append_kernel(")] \
        if "token_place(" in body else ""
    assert re.search(r"__ldcg\(tokens", body)
    assert not re.search(r"__ldg\((tokens|values)", body)


# ---- chains on the GPU --------------------------------------------------------------
def captured(fn):
    """fn recorded once: its launches follow one another without the host's pauses."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            fn()
    torch.cuda.current_stream().wait_stream(side)
    return g


@gpu
@pytest.mark.parametrize("B,V,dtype", [(1, 32768, torch.float32), (8, 262144, torch.float32),
                                       (8, 151936, torch.bfloat16), (200, 20000, torch.bfloat16)])
def test_append_after_a_filter_with_nothing_to_filter(B, V, dtype):
    """Greedy rows, and rows without a filter, leave the filter kernel at once;
    the tokens appended next are still those that the sampler before it wrote."""
    n = 12
    g = torch.Generator("cuda").manual_seed(B)
    x = [(torch.randn(B, V, generator=g, device="cuda") * 3).to(dtype) for _ in range(n)]
    T = torch.zeros(B, device="cuda")
    T[1::2] = 0.9
    seed = torch.arange(B, device="cuda")
    offset = torch.zeros(B, dtype=torch.int64, device="cuda")
    k = torch.where(T > 0, 0, 5).to(torch.int32)  # 0: no filter
    ws = gs.new_workspace(B)
    want = [gs.gumbel_argmax(y, T, seed, offset).cpu().numpy() for y in x]
    out = torch.full((n, B), -1, dtype=torch.int64, device="cuda")
    state = gs.new_logit_state(B, V, bias=False)
    warm = gs.new_logit_state(B, V, bias=False)
    gs.filtered_gumbel_argmax(x[0], T, seed, offset, top_k=k, out=out[0], workspace=ws)
    gs.history_append(warm, out[0])

    def steps():
        for i in range(n):
            gs.filtered_gumbel_argmax(x[i], T, seed, offset, top_k=k, out=out[i], workspace=ws)
            gs.history_append(state, out[i])

    graph = captured(steps)
    for _ in range(10):
        out.fill_(-1)
        gs.state_reset(state)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), np.stack(want))
        counts = np.zeros((B, V), np.int32)
        for w in want:
            np.add.at(counts, (np.arange(B), w), 1)
        assert np.array_equal(state.history[:, :V].cpu().numpy(), counts)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,V", [(1, 50257), (9, 33000), (90, 20001), (180, 9001)])
def test_draws_from_logits_processed_in_place(B, V, dtype):
    """Refill, constrain in place, draw, over and over without a pause: every
    sampler sees the logits that were just written, wherever rows start."""
    n = 6
    rng = np.random.default_rng([B, V])
    for pitch, shift in ((3, 1), ((-V) % 64, 0)):
        g = torch.Generator("cuda").manual_seed(V)
        src = [(torch.randn(B, V, generator=g, device="cuda") * 3).to(dtype) for _ in range(n)]
        words = (V + 31) // 32
        masks = [torch.from_numpy(rng.integers(-2**31, 2**31, (B, words)).astype(np.int32)).cuda()
                 for _ in range(n)]
        state = gs.new_logit_state(B, V)
        gs.bias_set(state, torch.arange(B, device="cuda") * 5 % V,
                    torch.full((B,), 9.0, device="cuda"))
        buf = torch.zeros(B * (V + pitch) + shift + 8, dtype=dtype, device="cuda")
        x = buf[shift:shift + B * (V + pitch)].view(B, V + pitch)[:, :V]
        T = torch.full((B,), 0.8, device="cuda")
        T[::3] = 0.0
        seed = torch.arange(B, device="cuda")
        zero = torch.zeros(B, dtype=torch.int64, device="cuda")
        three = torch.full((B,), 3, dtype=torch.int32, device="cuda")
        ws = gs.new_workspace(B)
        calls = [lambda o: gs.gumbel_argmax(x, T, seed, zero, out=o, workspace=ws),
                 lambda o: gs.constrained_gumbel_argmax(x, T, seed, zero, out=o, workspace=ws),
                 lambda o: gs.argmax(x, out=o, workspace=ws),
                 lambda o: gs.filtered_gumbel_argmax(x, T, seed, zero, top_k=three, out=o,
                                                     workspace=ws),
                 lambda o: gs.categorical(x, T, seed, zero, out=o)]
        for call in calls:
            want = []
            for s, m in zip(src, masks):
                x.copy_(s)
                gs.process_logits(x, state=state, mask=m, out=x)
                torch.cuda.synchronize()
                want.append(torch.full((B,), -5, dtype=torch.int64, device="cuda"))
                call(want[-1])
                torch.cuda.synchronize()
            for _ in range(3):
                got = torch.full((n, B), -5, dtype=torch.int64, device="cuda")
                for i in range(n):
                    x.copy_(src[i])
                    gs.process_logits(x, state=state, mask=masks[i], out=x)
                    call(got[i])
                assert torch.equal(got, torch.stack(want))


@gpu
def test_biases_of_the_tokens_and_values_just_written():
    """Lists that the kernel before wrote: the tokens a sampler drew, and
    constrained logits as values."""
    B, V, n = 40, 5000, 8
    g = torch.Generator("cuda").manual_seed(1)
    x = [torch.randn(B, V, generator=g, device="cuda") for _ in range(n)]
    ids = torch.arange(B, device="cuda")
    place, ends = ids.float(), torch.tensor([0, B], device="cuda")
    rows = torch.zeros(B, dtype=torch.int32, device="cuda")
    state = gs.new_logit_state(1, V)
    idx = torch.zeros(B, dtype=torch.int64, device="cuda")
    vals = torch.zeros(1, B, device="cuda")
    ws = gs.new_workspace(B)
    seen = []
    for y in x:
        gs.argmax(y, out=idx, workspace=ws)
        gs.bias_set(state, idx, place, offsets=ends)
        seen.append(state.bias[0].clone())
        gs.state_reset(state, slots=rows[:1])
        gs.process_logits(y[:1, :B], out=vals)
        gs.bias_set(state, ids, vals[0], offsets=ends)
        seen.append(state.bias[0].clone())
        gs.state_reset(state, slots=rows[:1])
    for i, y in enumerate(x):
        want = np.zeros(state.ld, np.float32)
        for j, t in enumerate(y.argmax(1).tolist()):  # the later value stays
            want[t] = j
        assert np.array_equal(seen[2 * i].cpu().numpy(), want)
        want[:] = 0
        want[:B] = y[0, :B].cpu().numpy()
        assert np.array_equal(seen[2 * i + 1].cpu().numpy(), want)
