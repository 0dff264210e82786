"""Which of a model's parameters are matrices whose updates are orthogonalised."""
import torch

from protein_folding_triangle_gb300 import layers


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(7, 32)
        self.bag = torch.nn.EmbeddingBag(5, 32)
        self.norm = layers.QKNorm(2, 16)
        self.shared = layers.QKNorm(2, 16, shared=True)
        self.rel = layers.RelativePosition(4, chains=True)
        self.ffn = layers.Transition(32, 64)
        self.out = torch.nn.Linear(32, 7)
        self.tied = torch.nn.Linear(32, 7, bias=False)
        self.tied.weight = self.embed.weight
        self.again = self.out
        self.w = torch.nn.Parameter(torch.zeros(3, 5))


def test_matrices_of_products_alone():
    m = Model()
    got = layers.matrix_parameters(m)
    want = [m.w, m.ffn.w_in, m.ffn.w_o, m.out.weight]
    assert [id(p) for p in got] == [id(p) for p in want]
    assert layers.matrix_parameters(m.norm) == [] and layers.matrix_parameters(m.rel) == []


class Rows(torch.nn.Module):
    NOT_MATRICES = ("rows",)

    def __init__(self):
        super().__init__()
        self.rows, self.w = (torch.nn.Parameter(torch.zeros(4, 4)) for _ in range(2))


def test_a_module_of_the_users():
    m = torch.nn.Sequential(Rows(), torch.nn.Linear(3, 4))
    assert [id(p) for p in layers.matrix_parameters(m)] == [id(m[0].w), id(m[1].weight)]
