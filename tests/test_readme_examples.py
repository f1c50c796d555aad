"""README's Python examples: log-probabilities that one example compares are of one distribution."""
import ast
import os
import re

README = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "README.md")
HEADS = ("grpo_logprobs", "grpo_logprobs_fwd", "grpo_ref_logprobs", "grpo_loss", "grpo_loss_fwd", "grpo_loss_bwd")


def examples():
    return re.findall(r"```python\n(.*?)```", open(README).read(), re.S)


def test_an_example_s_log_probabilities_have_the_same_options():
    """exp(lp - old) is 1 for unchanged weights only if both are formed by the same logit transform."""
    seen = 0
    for code in examples():
        given = {}
        for node in ast.walk(ast.parse(code)):
            if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute) and node.func.attr in HEADS:
                opts = [ast.unparse(k.value) for k in node.keywords if k.arg == "opts"]
                given.setdefault(opts[0] if opts else "none", []).append(node.func.attr)
                seen += 1
        assert len(given) <= 1, given
    assert seen >= 5
