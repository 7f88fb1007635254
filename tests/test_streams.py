"""Calls on another stream than the current one: what they allocate (scratch, results) belongs to that stream, and
results are kept from reuse while the caller's stream reads them."""
from __future__ import annotations

import contextlib
import types

import pytest
import torch

import sparse_moe_layer_07_b200 as moe
from sparse_moe_layer_07_b200 import expert_parallel, sharded
from synth import configs

from parity_util import LayerInputs

HOLD = 40_000_000  # clocks that a stream is held up: about 20 ms, a thousand times a launch


def test_allocations_are_made_under_the_stream(monkeypatch):
    made, current = [], ["here"]

    @contextlib.contextmanager
    def under(stream):
        current.append(stream.name)
        yield
        current.pop()

    class Like:
        dtype, shape = torch.float32, (3,)

        def new_empty(self, shape, dtype=None):
            made.append((current[-1], shape))
            return torch.empty(shape, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    side = types.SimpleNamespace(name="side", device=torch.device("cuda", 0))
    moe._empty((2,), torch.int32, Like(), None)
    moe._empty((2,), torch.int32, Like(), side)
    moe._empty_like(Like(), (3,), side)
    moe._empty_like(Like(), (4,), None)
    assert made == [("here", (2,)), ("side", (2,)), ("side", (3,)), ("here", (4,))]
    # functions of several steps run with their stream as the current one
    assert moe._on_stream(lambda a, stream=None: (a, current[-1], stream))(1, side) == (1, "side", None)
    assert moe._on_stream(lambda a, stream=None: (a, current[-1], stream))(1) == (1, "here", None)


def test_a_stream_of_another_device_is_refused():
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        moe._stream(other, torch.device("cuda", 0))


def _jobs():
    """name -> (call(stream) with neither scratch nor results given, bytes of what it allocates)."""
    w = configs.scaled(configs.WORKLOADS["mid_bf16"], name="streams", T=700, d=512, f=512, capacity_factor=4.0)
    L = LayerInputs(w)
    c, D = L.cfg, L.dev
    W = (D["wr"], D["wg"], D["wu"], D["wd"])
    idx, wts, lg = moe.router_topk(c, D["x"], D["wr"], want_logits=True)
    disp = moe.dispatch(c, D["x"], idx, wts)
    qw, q8 = moe.MxExperts(c, *W[1:]), moe.QuantizedExperts(c, *W[1:])
    h, y = moe.expert_ffn(c, disp["x_perm"], disp["offsets"], *W[1:], disp["row_scale"])
    off = torch.tensor([0, 100, 699], dtype=torch.int32, device="cuda")
    big = moe.Config(30000, 512, 512)
    blg = torch.randn((30000, 8), device="cuda")
    bidx = blg.topk(2, dim=1).indices.to(torch.int32)
    T, d, f, rows = 700, 512, 512, 1400
    codes, scales = moe.quantize_mx4(c, D["wg"])
    ck = torch.empty(moe.checkpoint_size_c8(c), dtype=torch.uint8, device="cuda")
    sc = torch.empty(moe.workspace_size_train_c8(c), dtype=torch.uint8, device="cuda")
    out2 = moe.layer_forward_train_c8(c, D["x"], *W, ck, sc)
    wst = torch.empty(moe.workspace_size_train(c), dtype=torch.uint8, device="cuda")
    moe.layer_forward_train(c, D["x"], *W, wst)
    torch.cuda.synchronize()
    act = T * d * 2
    return {
        "layer_forward_mx4": (lambda s: moe.layer_forward_mx4(c, D["x"], D["wr"], qw, stream=s),
                              (moe.workspace_size_mx4(c), act)),
        "expert_ffn_mx4": (lambda s: moe.expert_ffn_mx4(c, disp["x_perm"], disp["offsets"], qw, disp["row_scale"],
                                                       stream=s)[:int(disp["offsets"][8])],
                           (moe.expert_ffn_mx4_workspace_size(c), rows * d * 4)),
        "quantize_mx4": (lambda s: moe.quantize_mx4(c, D["wg"], stream=s), (4 * d * f, 4 * d * f // 16)),
        "dequantize_mx4": (lambda s: moe.dequantize_mx4(c, codes, scales, stream=s), (16 * d * f,)),
        "balance_loss": (lambda s: moe.balance_loss(c, lg, idx, seq_offsets=off, stream=s), (T * 32, 64, 512)),
        "balance_loss_large": (lambda s: moe.balance_loss(big, blg, bidx, stream=s),
                               (moe.balance_loss_workspace_size(big), 30000 * 32, 512)),
        "layer_backward_c8": (lambda s: moe.layer_backward_c8(c, D["x"], *W, out2, ck, sc, stream=s),
                              (8 * d * f * 2, act)),
        "layer_backward": (lambda s: moe.layer_backward(c, D["x"], *W, out2, wst, stream=s),
                           (8 * d * f * 4, act)),
        "layer_forward": (lambda s: moe.layer_forward(c, D["x"], *W, stream=s), (moe.workspace_size(c), act)),
        "layer_forward_w8": (lambda s: moe.layer_forward_w8(c, D["x"], D["wr"], q8, stream=s),
                             (moe.lib.moe_workspace_size_w8(c.ref), act)),
        "expert_down_combine": (lambda s: moe.expert_down_combine(c, h, disp["offsets"], D["wd"], disp["row_scale"],
                                                                 disp["perm"], stream=s),
                                (moe.lib.moe_expert_down_combine_workspace_size(c.ref), act)),
        "dispatch": (lambda s: {k: v for k, v in moe.dispatch(c, D["x"], idx, wts, stream=s).items()
                                if k in ("counts_kept", "slot_of")},
                     (moe.dispatch_workspace_size(c), rows * d * 2, rows * 4)),
        "router_topk": (lambda s: moe.router_topk(c, D["x"], D["wr"], want_logits=True, stream=s), (rows * 4, T * 32)),
        "combine": (lambda s: moe.combine(c, y, disp["slot_of"], stream=s), (act,)),
        "layer_forward_shard": (lambda s: sharded.layer_forward_shard(c, T, lambda n: n[None], 0, D["x"], *W, stream=s)[0],
                                (rows * d * 2, rows * d * 4, rows * f * 2, act)),
        "ep_forward_peers_local": (lambda s: expert_parallel.ep_forward_peers_local(c, [D["x"], D["x"]], *W, stream=s),
                                   (2 * rows * f * 2, act)),
    }


def _tensors(r):
    if isinstance(r, torch.Tensor):
        return [r]
    return [t for v in (r.values() if isinstance(r, dict) else r) if v is not None for t in _tensors(v)]


@pytest.fixture(scope="module")
def jobs():
    made = _jobs()
    return {k: (call, sizes, [t.clone() for t in _tensors(call(None))]) for k, (call, sizes) in made.items()}


NAMES = ("layer_forward_mx4", "expert_ffn_mx4", "quantize_mx4", "dequantize_mx4", "balance_loss", "balance_loss_large",
         "layer_backward_c8", "layer_backward", "layer_forward", "layer_forward_w8", "expert_down_combine", "dispatch",
         "router_topk", "combine", "layer_forward_shard", "ep_forward_peers_local")


def _same(got, want):
    got = _tensors(got)
    return len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_scratch_is_not_handed_out_before_the_call_ran(jobs, name):
    call, sizes, want = jobs[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    got = call(side)  # runs behind the hold; its scratch is dropped here
    taken = [torch.full((n,), 119, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(bool((t == 119).all()) for t in taken)
    assert _same(got, want) and moe.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_blocks_in_use_on_the_current_stream_are_not_written(jobs, name):
    call, sizes, want = jobs[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    used = [torch.full((n,), 5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda._sleep(HOLD)
    read = [u.clone() for u in used]  # behind the hold
    del used
    got = call(side)
    torch.cuda.synchronize()
    assert all(bool((r == 5).all()) for r in read)
    assert _same(got, want) and moe.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_results_stay_while_the_current_stream_reads_them(jobs, name):
    call, sizes, want = jobs[name]
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    got = _tensors(call(side))
    here.wait_stream(side)
    torch.cuda._sleep(HOLD)
    read = [t.clone() for t in got]  # behind the hold
    del got
    with torch.cuda.stream(side):  # takes the same sizes there and writes them
        for n in sizes:
            for _ in range(2):
                torch.full((n,), 119, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert _same(read, want) and moe.get_device_error() == 0
