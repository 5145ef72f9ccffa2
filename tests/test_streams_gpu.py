"""The recurrence's calls with stream=: the outputs and workspaces they allocate belong to that stream, and the
lengths they fetch are read there."""
import pytest
import torch

pytestmark = pytest.mark.gpu
H, D = 4, 128


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available()
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


def inputs(rows, slots, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    return {"qkv": randn(rows, 3 * H * D).to(torch.bfloat16), "g": randn(rows, H * D).to(torch.bfloat16), "b": randn(rows, H).to(torch.bfloat16),
            "A": 0.3 * randn(H), "dt": 0.1 * randn(H * D), "state": 0.05 * randn(slots, H, D, D),
            "index": torch.arange(slots, dtype=torch.int32, device="cuda")}


def calls(kda):
    """Every call that allocates, with outputs (and workspaces) of a megabyte or more."""
    x = inputs(4096, 4096, 1)
    few = inputs(2048, 8, 2)
    cu = torch.tensor([0, 700, 1400, 2048], dtype=torch.int32)
    cu_gpu = cu.cuda()
    mixed = torch.tensor([0, 1, 2, 2048], dtype=torch.int32)
    mixed_gpu = mixed.cuda()

    def common(i):
        return i["qkv"], i["g"], i["b"], i["A"], i["dt"], None, i["state"].clone(), i["index"]

    args, few_args = common(x), common(few)
    start, few_start = args[6].clone(), few_args[6].clone()
    table = torch.arange(4096, dtype=torch.int32, device="cuda").view(512, 8)

    def reset():
        args[6].copy_(start)
        few_args[6].copy_(few_start)

    return reset, {
        "gate": lambda s: kda.kda_gate(x["g"], x["b"], x["A"], x["dt"], stream=s),
        "packed_decode": lambda s: kda.kda_packed_decode(*args, stream=s)[:1],
        "spec_verify": lambda s: kda.kda_spec_verify(*args, 8, stream=s)[:1],
        "spec_verify_checkpoints": lambda s: kda.kda_spec_verify_checkpoints(*args[:7], table, 8, stream=s)[:1],
        "fused_decode": lambda s: kda.kda_fused_decode(*args, stream=s)[:1],
        "fused_spec_verify": lambda s: kda.kda_fused_spec_verify(*args, 8, stream=s)[:1],
        "chunk_prefill": lambda s: kda.kda_chunk_prefill(*few_args, cu_gpu, cu_seqlens_host=cu, stream=s)[:1],
        "mixed_batch": lambda s: kda.kda_mixed_batch(*few_args, mixed_gpu, 2, cu_seqlens_host=mixed, stream=s)[:1]}


@pytest.mark.parametrize("name", ["gate", "packed_decode", "spec_verify", "spec_verify_checkpoints", "fused_decode", "fused_spec_verify",
                                  "chunk_prefill", "mixed_batch"])
def test_what_a_call_allocates_belongs_to_its_stream(kda, name):
    reset, all_calls = calls(kda)
    call, side = all_calls[name], torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    reset()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    blocks = {t.data_ptr(): t.nbytes for t in out if t.nbytes >= 1 << 20}
    assert blocks
    del out
    here = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in blocks.values()]
    with torch.cuda.stream(side):
        there = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in blocks.values()]
    assert not {t.data_ptr() for t in here} & set(blocks)
    assert {t.data_ptr() for t in there} == set(blocks)


@pytest.mark.parametrize("name", ["chunk_prefill", "mixed_batch"])
def test_a_workspace_is_not_handed_out_while_it_is_used(kda, name):
    """The workspace is dropped when the call returns, with its kernels still waiting on a busy stream; what is
    allocated and written on the current stream meanwhile must not be its memory."""
    reset, all_calls = calls(kda)
    call, side = all_calls[name], torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    reset()
    busy = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        for i in range(40):
            busy.fill_(i)
    out = call(side)
    junk = [torch.full((n << 20,), 0x7F, dtype=torch.uint8, device="cuda") for n in (1, 2, 4, 8, 16, 32, 64)]
    torch.cuda.synchronize()
    assert len(junk) == 7 and all(torch.equal(a, b) for a, b in zip(want, out))


def test_lengths_are_read_on_the_stream(kda):
    """cu_seqlens written on a busy stream and fetched by a call on it, with no host copy given."""
    x = inputs(256, 4, 3)
    state = x["state"].clone()
    values = torch.tensor([0, 100, 200, 256], dtype=torch.int32).cuda()
    args = (x["qkv"], x["g"], x["b"], x["A"], x["dt"], None)
    want, _ = kda.kda_chunk_prefill(*args, x["state"], x["index"], values)
    cu, busy, side = torch.zeros_like(values), torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(40):
            busy.fill_(i)
        cu.copy_(values)
    got, _ = kda.kda_chunk_prefill(*args, state, x["index"], cu, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(state, x["state"])
