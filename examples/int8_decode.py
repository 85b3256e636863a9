"""Scores a prompt and decodes greedily with INT8 weights.

A small language model without attention (embedding, a gated feed-forward block with a residual,
an LM head; random weights), run entirely through the library:

  weights   qw_quantize_int8 of their BF16 rows: codes [N][K] and a scale per output channel
  block     qgemm_int8_gated (tokens quantised inside the call), then qgemm_int8 back to the model's
            width
  head      the tokens quantised once by qw_quantize_int8, then qgemm_int8 of codes with FP32 logits
  answer    qw_logprobs: log probability and rank of each next token, entropy, top alternatives

A prompt runs as one batch; decoding runs one token at a time, the step captured once in a CUDA graph
and replayed.

    python examples/int8_decode.py --vocab 32000 --hidden 4096 --inner 14336 --prompt 512 --new 32
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_qw_repack_gb300 import qw as Q  # noqa: E402


def quantise_rows(w):
    """BF16 [rows][K] -> INT8 codes and FP32 scales of the rows."""
    codes = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    scale = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
    Q.qw_quantize_int8(w, w.stride(0), w.shape[0], w.shape[1], codes, scale)
    return codes, scale


class Model:
    def __init__(self, vocab, hidden, inner, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rows(n, k, std):
            return (torch.randn(n, k, generator=g, device=device) * std).to(torch.bfloat16)

        self.vocab, self.hidden, self.inner, self.device = vocab, hidden, inner, device
        self.embedding = rows(vocab, hidden, 1.0)
        self.gate_up = quantise_rows(rows(2 * inner, hidden, hidden ** -0.5))
        self.down = quantise_rows(rows(hidden, inner, inner ** -0.5))
        self.down_bias = rows(1, hidden, 0.1)[0]
        self.head = quantise_rows(rows(vocab, hidden, 4 * hidden ** -0.5))

    def session(self, tokens, top):
        return Session(self, tokens, top)


class Session:
    """Buffers for `tokens` tokens at a time, and the calls on them."""

    def __init__(self, model, tokens, top):
        m, dev = model, model.device
        self.model, self.tokens, self.top = m, tokens, top

        def new(*shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.ids = torch.zeros(tokens, dtype=torch.int32, device=dev)  # what is read
        self.next = torch.zeros(tokens, dtype=torch.int32, device=dev)  # what is scored
        self.y = new(tokens, m.inner, dtype=torch.bfloat16)
        self.h = new(tokens, m.hidden, dtype=torch.bfloat16)
        self.codes = new(tokens, m.hidden, dtype=torch.int8)
        self.scale = new(tokens, dtype=torch.float32)
        self.logits = new(tokens, m.vocab, dtype=torch.float32)
        self.logprob = new(tokens, dtype=torch.float32)
        self.rank = new(tokens, dtype=torch.int32)
        self.entropy = new(tokens, dtype=torch.float32)
        self.top_ids = new(tokens, top, dtype=torch.int32)
        self.top_logprobs = new(tokens, top, dtype=torch.float32)
        size = Q.qgemm_int8_workspace_size
        self.ws_bytes = max(size(Q.QW_A_BF16, tokens, 2 * m.inner, m.hidden),
                            size(Q.QW_A_BF16, tokens, m.hidden, m.inner),
                            size(Q.QW_A_INT8_TOKEN, tokens, m.vocab, m.hidden))
        self.workspace = new(max(self.ws_bytes, 1), dtype=torch.uint8)
        self.error = Q.new_error_flag()

    def step(self):
        """ids -> logits and the answer about `next`, on the current stream."""
        m, T = self.model, self.tokens
        ws = (self.workspace, self.ws_bytes, self.error)
        x = m.embedding.index_select(0, self.ids)
        Q.qgemm_int8_gated(Q.QW_A_BF16, x, m.hidden, None, *m.gate_up, None, self.y, m.inner, T,
                           m.inner, m.hidden, *ws)
        Q.qgemm_int8(Q.QW_A_BF16, self.y, m.inner, None, *m.down, m.down_bias, Q.QW_T_BF16, self.h,
                     m.hidden, T, m.hidden, m.inner, *ws)
        x = x + self.h
        Q.qw_quantize_int8(x, m.hidden, T, m.hidden, self.codes, self.scale, self.error)
        Q.qgemm_int8(Q.QW_A_INT8_TOKEN, self.codes, m.hidden, self.scale, *m.head, None, Q.QW_T_F32,
                     self.logits, m.vocab, T, m.vocab, m.hidden, *ws)
        Q.qw_logprobs(Q.QW_T_F32, self.logits, m.vocab, T, m.vocab, self.next, self.top,
                      self.logprob, self.rank, self.entropy, self.top_ids, self.top_logprobs,
                      self.error)

    def check(self):
        assert Q.qw_read_error(self.error) == Q.QW_OK


def score(model, prompt, top=5):
    """Log probability and rank of each token of the prompt after the first."""
    s = model.session(len(prompt) - 1, top)
    s.ids.copy_(prompt[:-1])
    s.next.copy_(prompt[1:])
    s.step()
    s.check()
    return s


def decode(model, first, count, top=5, graph=True):
    """Greedy continuation of the token `first`: ids and their log probabilities."""
    s = model.session(1, top)
    s.ids.fill_(int(first))
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.step()  # (loads the kernels before the capture)
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            s.step()
            s.ids.copy_(s.top_ids[:, 0])
    ids, logprobs = [], []
    for _ in range(count):
        if graph:
            captured.replay()
        else:
            s.step()
            s.ids.copy_(s.top_ids[:, 0])
        ids.append(s.top_ids[0, 0].clone())
        logprobs.append(s.top_logprobs[0, 0].clone())
    s.check()
    return torch.stack(ids), torch.stack(logprobs)


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("vocab", 32000), ("hidden", 4096), ("inner", 14336), ("prompt", 512),
                        ("new", 32), ("top", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    model = Model(a.vocab, a.hidden, a.inner)
    prompt = torch.randint(a.vocab, (a.prompt,), device="cuda", dtype=torch.int32)
    s = score(model, prompt, a.top)
    print(f"prompt of {a.prompt} tokens: mean log probability {s.logprob.mean().item():.3f}, "
          f"mean rank {s.rank.float().mean().item():.0f}, "
          f"mean entropy {s.entropy.mean().item():.3f}")
    ids, logprobs = decode(model, prompt[-1], a.new, a.top)
    print("continuation:", " ".join(f"{i}({p:.2f})" for i, p in zip(ids.tolist(), logprobs.tolist())))


if __name__ == "__main__":
    main()
