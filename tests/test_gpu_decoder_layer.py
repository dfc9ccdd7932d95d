"""A decoder layer's generation step out of the library's calls alone:

  norm -> qkv -> cache append -> attention -> o_proj -> norm with the residual
  -> gate_up -> SiLU -> down

on the W4A16 path (fp16 between the layers) and on the W4A8 path (the norms
and the SiLU write the E4M3 codes and scales that awq_w4a8_gemm takes). Every
stage is checked against its formula in fp64 on the inputs it was given, with
the tolerances of the stages' own tests; the whole step captured into a graph
gives the same bits."""
import numpy as np
import pytest
import torch

import awq_synth
import oracle
import weight_only_bit_awq_b200 as awq
from gpu_helpers import check_close, gpu_pack, host, packed_to_host
from test_gpu_kv8 import Batch, append_model, same_cache
from test_gpu_norm_act import EPS, check_fp16, check_fp8, fp32_slack, norm_ref, silu_ref

pytestmark = pytest.mark.gpu

HID, FF, HQ, HKV, D = 512, 1024, 8, 2, 64


class Layer:
    def __init__(self, fp8):
        self.fp8 = fp8
        self.packed = {}
        for name, N, K in (("qkv", (HQ + 2 * HKV) * D, HID), ("o", HID, HQ * D), ("gate_up", 2 * FF, HID), ("down", HID, FF)):
            dev = gpu_pack(awq_synth.matrix_f16(awq_synth.key(0, 77, f"layer/{name}"), N, K, 0.04))
            e = awq.awq_fp8_row_exponents(dev[1], K, N)
            self.packed[name] = (N, K, dev, e, packed_to_host(*dev))
        g = torch.Generator(device="cuda").manual_seed(3)
        self.w1, self.w2 = ((1 + 0.2 * torch.randn(HID, generator=g, device="cuda")).half() for _ in "12")
        need = max(awq.awq_workspace_bytes(M, p[1], p[0]) for p in self.packed.values() for M in range(1, 33))
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def linear(self, name, x):
        N, K, dev, e, _ = self.packed[name]
        if isinstance(x, tuple):
            return awq.awq_w4a8_gemm(x[0], x[1], *dev, e, N, self.ws)
        return awq.awq_linear(x, *dev, N, self.ws)

    def step(self, x, bt):
        """One step; every intermediate result, by name."""
        s = {"x": x}
        norm = awq.awq_rmsnorm_fp8 if self.fp8 else awq.awq_rmsnorm
        s["n1"] = norm(x, self.w1, EPS)
        s["qkv"] = self.linear("qkv", s["n1"])
        q, k, v = s["qkv"].split([HQ * D, HKV * D, HKV * D], dim=1)
        bt.q, bt.k, bt.v = q.unflatten(1, (HQ, D)), k.unflatten(1, (HKV, D)), v.unflatten(1, (HKV, D))
        bt.append()
        s["att"] = bt.attend()
        s["o"] = self.linear("o", awq.awq_fp8_quantize_x(s["att"]) if self.fp8 else s["att"])
        got = norm(s["o"], self.w2, EPS, residual=x)
        s["n2"], s["h"] = (got[:2], got[2]) if self.fp8 else got
        s["gate_up"] = self.linear("gate_up", s["n2"])
        s["act"] = awq.awq_silu_mul_fp8(s["gate_up"]) if self.fp8 else awq.awq_silu_mul(s["gate_up"])
        s["down"] = self.linear("down", s["act"])
        return s

    def check_linear(self, name, x, y):
        N, K, _, e, hp = self.packed[name]
        if isinstance(x, tuple):
            ref, b = oracle.fp8_linear(host(x[0], np.uint8), host(x[1], np.float32), *hp, host(e, np.int8), N, K)
        else:
            ref, b = oracle.linear(host(x, np.float16), *hp, N, K)
        check_close(host(y, np.float16), ref, b, name)

    def check(self, s, bt):
        def act(got, ref, rel, what):
            check_fp8(*got, ref, rel, what) if isinstance(got, tuple) else check_fp16(got, ref, rel, what)

        act(s["n1"], norm_ref(s["x"], self.w1, EPS), fp32_slack(HID), "n1")
        self.check_linear("qkv", s["n1"], s["qkv"])
        ref, tol = bt.attention_ref()
        assert ((s["att"].double() - ref).abs() <= tol).all()
        self.check_linear("o", awq.awq_fp8_quantize_x(s["att"]) if self.fp8 else s["att"], s["o"])
        assert torch.equal(s["h"], (s["o"].float() + s["x"].float()).half())
        act(s["n2"], norm_ref(s["o"], self.w2, EPS, s["x"]), fp32_slack(HID), "n2")
        self.check_linear("gate_up", s["n2"], s["gate_up"])
        act(s["act"], silu_ref(s["gate_up"]), (float(s["gate_up"].abs().max()) + 16) * 2.0 ** -23, "act")
        self.check_linear("down", s["act"], s["down"])
        assert awq.awq_get_status(self.ws) == awq.AWQ_OK and bt.status() == awq.AWQ_OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 1, 0, 5]])
def test_generation_step(fp8, new):
    layer = Layer(fp8)
    lens = [new[0], 70, 40, 130]
    bt = Batch(new, lens, HQ, HKV, D, 32, seed=20, empty=True)
    x = torch.randn(sum(new), HID, generator=bt.g, device="cuda").half()
    for _ in range(3):
        before = [t.clone() for t in bt.cache]
        s = layer.step(x, bt)
        same_cache(bt.cache, append_model(bt, before))
        layer.check(s, bt)
        x = (s["down"].float() + s["h"].float()).half()
        # the next tokens; the sequences grow
        bt.n = [n + t for n, t in zip(bt.n, new)]
        width = bt.table.shape[1]
        if max(bt.n) > width * bt.block:
            break
        bt.lens = torch.tensor(bt.n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
def test_generation_step_in_a_graph(fp8):
    layer = Layer(fp8)
    bt = Batch([1] * 5, [33, 64, 1, 100, 17], HQ, HKV, D, 32, seed=21)
    x = torch.randn(5, HID, generator=bt.g, device="cuda").half()
    keep = [t.clone() for t in bt.cache]
    want = layer.step(x, bt)
    cache = [t.clone() for t in bt.cache]
    for t, k in zip(bt.cache, keep):
        t.copy_(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(x, bt)
    for _ in range(3):
        for t, k in zip(bt.cache, keep):
            t.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            for a, b in zip(*(v if isinstance(v, tuple) else (v,) for v in (got[name], want[name]))):
                assert torch.equal(a, b), name
        same_cache(bt.cache, [t.cpu() for t in cache])
    assert bt.status() == awq.AWQ_OK and awq.awq_get_status(layer.ws) == awq.AWQ_OK


def test_two_batches_at_once_on_two_streams():
    # different caches and workspaces, one stream each, many calls in flight
    bts = [Batch([1] * 6, [900 + 300 * i for i in range(6)], 32, 8, 128, 64, seed=s) for s in (30, 31)]
    want = []
    for bt in bts:
        bt.append()
        want.append(bt.attend().clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for bt, st, ys in zip(bts, streams, got):
            with torch.cuda.stream(st):
                bt.append()
                bt.attend(y=ys[i])
    torch.cuda.synchronize()
    for ys, w, bt in zip(got, want, bts):
        assert all(torch.equal(y, w) for y in ys)
        assert bt.status() == awq.AWQ_OK
