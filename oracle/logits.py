"""Oracle: the target logits as served, with every request's own settings.

TEST INFRASTRUCTURE ONLY (see the package docstring).

"Speculative Decoding" (atlas), "Greedy, sampling and the real sampler": p must include the
transforms actually served.  Readings (the pages give no formulas): repetition r over prompt and
text, l / r or l r; frequency f and presence p over the text, l - f n - p; biases added; ids that
a grammar's mask forbids are -inf.  A row's text is the history behind the prompt and the block
tokens in front of it (a chain's drafts, a tree node's ancestors and the node).
"""
import numpy as np


def process(logits, history=None, prompt_len=None, block_tokens=None, parent=None,
            repetition=None, frequency=None, presence=None, bias_ids=None, bias=None, mask=None,
            mask_row=None, fp=np.float64):
    """logits [B, R, V]; every array as the call takes it (None: not given).  fp: the arithmetic,
    float32 for the served one, step by step."""
    y = np.array(logits, dtype=fp, copy=True)
    B, R, V = y.shape
    for b in range(B):
        for i in range(R):
            prompt, count = set(), {}
            for at, t in enumerate([] if history is None else history[b]):
                if 0 <= t < V:
                    if prompt_len is not None and at < prompt_len[b]:
                        prompt.add(int(t))
                    else:
                        count[int(t)] = count.get(int(t), 0) + 1
            v = i
            while v > 0 and block_tokens is not None:
                t = int(block_tokens[b][v if parent is not None else v - 1])
                if 0 <= t < V:
                    count[t] = count.get(t, 0) + 1
                u = int(parent[b][v]) if parent is not None else v - 1
                v = u if u < v else 0
            row = y[b, i]
            if repetition is not None:
                for t in prompt | set(count):
                    r = fp(repetition[b])
                    row[t] = row[t] / r if row[t] > 0 else row[t] * r
            for t, n in count.items():
                if frequency is not None:
                    row[t] = row[t] - fp(frequency[b]) * fp(n)
                if presence is not None:
                    row[t] = row[t] - fp(presence[b])
            if bias_ids is not None:
                total = {}
                for t, x in zip(bias_ids[b], bias[b]):
                    if 0 <= t < V:
                        total[int(t)] = fp(total.get(int(t), fp(0)) + fp(x))
                for t, x in total.items():
                    row[t] = row[t] + x
            if mask is not None:
                m = int(mask_row[b][i]) if mask_row is not None else b * R + i
                if 0 <= m < len(mask):
                    for t in range(V):
                        if not int(mask[m][t // 32]) >> (t % 32) & 1:
                            row[t] = -np.inf
    return y
