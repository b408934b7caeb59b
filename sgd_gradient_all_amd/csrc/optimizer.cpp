// optimizer.cpp -- the registry of the optimizers' live handles.
#include "optimizer_internal.h"

#include <set>

namespace ddl {
namespace {
std::mutex g_mu;
// never destroyed: handles may outlive static destruction
std::set<const void *> &g_live = *new std::set<const void *>;
}  // namespace

void register_handle(const void *h) {
    std::lock_guard<std::mutex> lk(g_mu);
    g_live.insert(h);
}

bool unregister_handle(const void *h) {
    std::lock_guard<std::mutex> lk(g_mu);
    return g_live.erase(h) == 1;
}

bool hold_handle(const void *h, std::unique_lock<std::mutex> &lk) {
    lk = std::unique_lock<std::mutex>(g_mu);
    return g_live.count(h) == 1;
}

}  // namespace ddl
