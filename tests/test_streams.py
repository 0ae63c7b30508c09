"""Memory that the allocating wrappers hand out for work on another stream belongs to that stream in torch's allocator."""
import contextlib

import pytest
import torch

import attention_quantized_kv_split_gb300 as qda


def wrappers(device):
    """Every call that allocates, with the foreign calls left out where there is no GPU to make them on."""
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
    pool = qda.PagedKV(3, 2, 16, 64, 32, 4, torch.bfloat16, device=device)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=device)
    flat = qda.QuantizedKV.empty([5], 2, 64, 32, 4, torch.bfloat16, device=device)
    for t in (flat.ks, flat.kb, flat.vs, flat.vb):
        t.zero_()
    rows = torch.zeros(1, 2, 2, 64, device=device).transpose(1, 2)   # not contiguous: copied by the call
    return {
        "step_tables": lambda s: pool.step_tables(i32(1), i32(1) + 2, i32(1, 2) - 1, torch.arange(3, dtype=torch.int32, device=device),
                                                  4, stream=s)["slots"],
        "attend": lambda s: pool.attend(q, i32(2) + torch.tensor([0, 2], dtype=torch.int32, device=device), i32(1) + 2,
                                        i32(1, 1), 2, stream=s),
        "decode_attention": lambda s: qda.decode_attention(q[:1], flat, stream=s),
        "append": lambda s: flat.append(rows, rows, stream=s).kp,
    }


@pytest.mark.parametrize("name", ["step_tables", "attend", "decode_attention", "append"])
def test_allocates_in_the_streams_context(name, monkeypatch):
    inside, seen = [], []

    @contextlib.contextmanager
    def on(stream, device):
        inside.append(stream)
        yield
        inside.pop()

    call = wrappers("cpu")[name]
    monkeypatch.setattr(qda, "_on", on)
    for f in ("qdecode_paged_map", "qdecode_paged_attn", "qdecode_attn"):
        monkeypatch.setattr(qda, f, lambda *a, **k: a[0] if name == "step_tables" else a[7])
    monkeypatch.setattr(qda, "lib", lambda: type("L", (), {"qdecode_cache_append": staticmethod(lambda *a: 0)}))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(list(inside)), empty(*a, **k))[1])
    call(77)
    assert seen and all(s == [77] for s in seen)


def test_the_current_stream_needs_no_context():
    assert isinstance(qda._on(None, "cpu"), contextlib.nullcontext)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["step_tables", "attend", "decode_attention", "append"])
def test_blocks_of_the_current_stream_are_not_taken(name, handle):
    call, s = wrappers("cuda")[name], torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    first = call(None)   # a block of this size of the current stream's, given back
    ref, at, size = first.clone(), first.data_ptr(), first.untyped_storage().nbytes()
    del first
    torch.cuda.synchronize()
    got = call(s.cuda_stream if handle else s)
    s.synchronize()
    assert not at <= got.data_ptr() < at + size
    assert torch.equal(got.view(torch.int16), ref.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [0, 1])
def test_the_default_streams_handle(stream):
    call = wrappers("cuda")["attend"]
    ref = call(None)
    assert torch.equal(call(stream), ref)
