// launch_turn.h -- calls of several kernels that share a workspace, from
// several host threads: one call's kernels follow each other on the stream.
#pragma once

#include <condition_variable>
#include <mutex>
#include <new>

namespace qmoe {

// Held over a call's launches.  Two threads that share a stream and a workspace
// must not put one call's second kernel behind the other's first; calls with
// other workspaces do not wait for each other: a launch blocks while its stream
// is full, and what that stream waits for may be another device's call.  (Other
// threads' launches on the same device the driver itself keeps waiting then:
// 1.5 s behind a full stream with one lock over all launches and with this.)
// key: the workspace, null: nothing to keep together.
class LaunchTurn {
public:
    explicit LaunchTurn(const void *key) : key_(key), next_(nullptr)
    {
        if (!key_)
            return;
        std::unique_lock<std::mutex> lock(mu());
        while (taken(key_))
            left().wait(lock);
        next_ = head();
        head() = this;
    }
    ~LaunchTurn()
    {
        if (!key_)
            return;
        {
            std::lock_guard<std::mutex> lock(mu());
            LaunchTurn **p = &head();
            while (*p != this)
                p = &(*p)->next_;
            *p = next_;
        }
        left().notify_all();
    }
    LaunchTurn(const LaunchTurn &) = delete;
    LaunchTurn &operator=(const LaunchTurn &) = delete;

private:
    static bool taken(const void *key)
    {
        for (const LaunchTurn *t = head(); t; t = t->next_)
            if (t->key_ == key)
                return true;
        return false;
    }
    // never destroyed: a thread may still wait here when the process ends, and
    // destroying a condition waits for its waiters
    template <class T>
    static T &kept()
    {
        alignas(T) static unsigned char room[sizeof(T)];
        static T *t = new (room) T;
        return *t;
    }
    static std::mutex &mu() { return kept<std::mutex>(); }
    static std::condition_variable &left() { return kept<std::condition_variable>(); }
    static LaunchTurn *&head()   // the calls that are launching, on their threads' stacks
    {
        static LaunchTurn *h = nullptr;
        return h;
    }

    const void *key_;
    LaunchTurn *next_;
};

}  // namespace qmoe
